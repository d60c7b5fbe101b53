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

// A row array as the loads see it: 16-byte pieces may be taken from [lo, hi) only.
struct RowSrc {
  const uint8_t *base, *lo, *hi;  // lo, hi: 16-byte aligned, inside the array
  long long ld;                   // bytes
  int cols, aligned;              // aligned: every row starts and ends at 16 bytes
};

struct TcArgs {
  FfnArgs f;
  const uint8_t* img;   // packed weights, chunk after chunk
  int nch, stage_bytes; // chunks; bytes of one
  int nst, ng;          // weight stages in shared memory; groups
  int dp, op;           // D and O rounded up to 16
  RowSrc x, dy;
  int out_aligned;      // y's or dx's rows start and end at 16 bytes
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

// 2^v and 1 / v of the special function unit: relative error below 2^-22 each, for results that are
// rounded to 8 or 11 bits. The unit takes one value per lane group and cycle (16 an SM), which is
// what bounds these kernels at narrow widths, so four reciprocals are taken as one: with
// r = 1 / (p0 p1 p2 p3) each is r times the product of the other three.
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
__device__ __forceinline__ void rcp4(const float (&p)[4], float (&r)[4]) {
  const float m01 = p[0] * p[1], m23 = p[2] * p[3];
  const float i = rcp_fast(m01 * m23);
  const float i01 = i * m23, i23 = i * m01;
  r[0] = i01 * p[1];
  r[1] = i01 * p[0];
  r[2] = i23 * p[3];
  r[3] = i23 * p[2];
}

// act and its slope for four values. MODE-independent; without SLOPE the slope is not formed.
//   silu: s = 1 / (1 + 2^t), t = -a log2 e held at 31 so that four factors stay finite: s is then
//         never below 2^-31, which differs from the true value by less than an fp32 step of 1/128.
//   gelu: Phi by Abramowitz and Stegun 7.1.26 (erfc at z = |a| / sqrt 2, absolute error 0.75e-7 in
//         Phi), z held at 10 where Phi(-|a|) has long become zero; one power e^{-a^2/2} serves Phi
//         and the density.
// An argument that is no number gives no number: both are multiplied by a, or built from it.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void act4(const float* a, float* f, float* slope) {
  float p[4], r[4];
  if (ACT == SPLAT_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = 1.0f + ex2_fast(fminf(a[i] * -1.4426950408889634f, 31.0f));
    rcp4(p, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i] * r[i];
      if (SLOPE) slope[i] = fmaf(f[i], 1.0f - r[i], r[i]);
    }
  } else {
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = fminf(fabsf(a[i]) * 0.70710678118654752f, 10.0f);
      p[i] = fmaf(0.3275911f, z[i], 1.0f);
    }
    rcp4(p, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = ex2_fast(z[i] * z[i] * -1.4426950408889634f);
      float q = fmaf(0.5307027145f, r[i], -0.7265760135f);  // half the published coefficients
      q = fmaf(q, r[i], 0.7107068705f);
      q = fmaf(q, r[i], -0.142248368f);
      q = fmaf(q, r[i], 0.127414796f);
      q = q * r[i] * e;
      const float c = a[i] >= 0.0f ? 1.0f - q : q;
      f[i] = a[i] * c;
      if (SLOPE) slope[i] = fmaf(a[i] * 0.3989422804014327f, e, c);
    }
  }
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

// A group takes its tile of rows [r0, r0 + 128) with eight threads to a row: thread t has piece
// t & 7 (16 bytes, 8 elements) of each 64-column block of rows t / 8 + 32 j. The swizzle and a
// row's offset from 16-byte alignment are then the same for all four j. Rows >= M are zeros, and
// so are elements behind a row's end up to the next multiple of 16 (the MMAs' step; nothing reads
// what lies behind).

// aligned rows: one 64-column block's loads, started and then stored
__device__ __forceinline__ void fetch_rows(const RowSrc& s, int block, long long r0, long long M,
                                           int tid, uint4 (&v)[4]) {
  const int c = block * 8 + (tid & 7);
  const long long r = r0 + (tid >> 3);
  const uint8_t* p = s.base + r * s.ld + c * 16;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = make_uint4(0u, 0u, 0u, 0u);
    if (c * 8 < s.cols && r + 32 * j < M)
      v[j] = __ldg(reinterpret_cast<const uint4*>(p + 32 * j * s.ld));
  }
}

__device__ __forceinline__ uint8_t* piece_at(uint8_t* dst, int block, int tid) {
  return dst + block * 16384 + (tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) << 4);
}

__device__ __forceinline__ void store_rows(int block, int tid, const uint4 (&v)[4], uint8_t* dst) {
  uint8_t* q = piece_at(dst, block, tid);
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(q + j * 4096) = v[j];
}

// any other rows: the aligned 16-byte pieces around each piece (odd widths start anywhere), shifted
// into place. Pieces that reach over the array's ends are gathered element by element.
__device__ __forceinline__ void gather_rows(const RowSrc& s, int block, long long r0, long long M,
                                            int tid, uint8_t* dst) {
  const int c = block * 8 + (tid & 7);
  const long long r = r0 + (tid >> 3);
  const uint8_t* p = s.base + r * s.ld + c * 16;
  const int n = min(8, s.cols - c * 8);  // elements wanted
  const uint32_t off = (uint32_t)(uintptr_t)p & 15u;
  const bool two = (int)off + 2 * n > 16;
  uint8_t* q = piece_at(dst, block, tid);
#pragma unroll
  for (int j = 0; j < 4; ++j, p += 32 * s.ld) {
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (n > 0 && r + 32 * j < M) {
      const uint8_t* a = p - off;
      if (a >= s.lo && a + (two ? 32 : 16) <= s.hi) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(a));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        if (two) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(a + 16));
          w[4] = u.x, w[5] = u.y, w[6] = u.z, w[7] = u.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (2 * k >= (int)off && 2 * k < (int)off + 2 * n)
            w[k >> 1] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(a + 2 * k))
                         << ((k & 1) * 16);
      }
    }
    if (off & 4u) {
#pragma unroll
      for (int k = 0; k < 7; ++k) w[k] = w[k + 1];
    }
    if (off & 8u) {
#pragma unroll
      for (int k = 0; k < 5; ++k) w[k] = w[k + 2];
    }
    const uint32_t sh = (off & 2u) * 8u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = __funnelshift_r(w[k], w[k + 1], sh);
      if (n < 8) w[k] = n >= 2 * k + 2 ? w[k] : n == 2 * k + 1 ? w[k] & 0xFFFFu : 0u;
    }
    *reinterpret_cast<uint4*>(q + j * 4096) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// the rows' lines on their way into L2
__device__ __forceinline__ void prefetch_row(const RowSrc& s, long long r, long long M) {
  if (r >= M) return;
  const uint8_t* p = s.base + r * s.ld;
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p + s.cols * 2 - 2));
}

// One 64-column block of results (columns col0 ..) from shared memory to a row array: aligned rows
// in 16-byte pieces, others element by element with neighbouring lanes on neighbouring elements.
__device__ __forceinline__ void write_rows(const uint8_t* src, uint8_t* base, long long ld,
                                           int aligned, int col0, int cols, long long r0,
                                           long long M, int tid) {
  if (aligned) {
    const int c = tid & 7;
    const long long r = r0 + (tid >> 3);
    if (col0 + c * 8 >= cols) return;
    const uint8_t* q = src + (tid >> 3) * 128 + ((c ^ ((tid >> 3) & 7)) << 4);
    uint8_t* p = base + r * ld + col0 * 2 + c * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r + 32 * j < M)
        *reinterpret_cast<uint4*>(p + 32 * j * ld) = *reinterpret_cast<const uint4*>(q + j * 4096);
  } else {
    const int lane = tid & 31;
    const int n = min(64, cols - col0);
    for (int r = tid >> 5; r < kTile && r0 + r < M; r += kGroupThreads / 32)
      for (int e = lane; e < n; e += 32)
        *reinterpret_cast<uint16_t*>(base + (r0 + r) * ld + (col0 + e) * 2) =
            *reinterpret_cast<const uint16_t*>(src + r * 128 + (((e >> 3) ^ (r & 7)) << 4) +
                                               (e & 7) * 2);
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
      mbar_init(empty(s), p.ng);
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
    // (the whole warp waits, one lane issues)
    if (nt > 0) {
      const int kx = p.dp >> 4, ko = p.op >> 4;
      const uint32_t id_gu = idesc(BF, WR, false, false), id_dh = idesc(BF, 64, false, true);
      const uint32_t id_y = idesc(BF, p.op, false, false), id_dx = idesc(BF, p.dp, false, true);
      const uint32_t id_wx = idesc(BF, p.dp, true, true), id_wy = idesc(BF, p.op, true, true);
      // descriptors count in 16 bytes: a step of 16 along K is 2 in a K-major tile (4 steps to a
      // 64-column block), 128 in an MN-major one; weights' blocks have WR rows
      constexpr uint32_t kBlk = 16384 >> 4, kWBlk = WR * 128 >> 4;
      const uint32_t x0 = sbase + groups0, y0 = x0 + nbx * 16384;
      const uint32_t h0 = x0 + (nbx + (MODE == kFwd ? 0 : nby)) * 16384;
      const uint32_t dx_k = desc_lo(x0, 16), dy_k = desc_lo(y0, 16), dh_k = desc_lo(h0, 16);
      const uint32_t dx_mn = desc_lo(x0, 16384), dy_mn = desc_lo(y0, 16384), dh_mn = desc_lo(h0, 16384);
      const uint32_t dw_k = desc_lo(sbase, 16), dw_mn = desc_lo(sbase, WR * 128);
      const uint32_t dd_k = desc_lo(sbase + nbx * WR * 128, 16);
      const uint32_t gs = gbytes >> 4, ss = p.stage_bytes >> 4;
      // A|U (and dH) of group g from stage s
      auto first_product = [&](int g, int s) {
        if (elect_one()) {
          const uint32_t d = tmem + g * tg;
          const uint32_t a = dx_k + g * gs, b = dw_k + s * ss;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < kx)
              mma(d, a + (k >> 2) * kBlk + (k & 3) * 2, b + (k >> 2) * kWBlk + (k & 3) * 2, id_gu,
                  k > 0);
          if (MODE != kFwd) {
            const uint32_t ay = dy_k + g * gs, bd = dd_k + s * ss;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < ko)
                mma(d + 128, ay + (k >> 2) * kBlk + (k & 3) * 2, bd + k * 128, id_dh, k > 0);
          }
          commit(gu_full(g));
        }
        __syncwarp();
      };
      auto second_product = [&](int g, int s, bool add, bool begun, bool last_chunk, bool ring,
                                bool last) {
        if (elect_one()) {
          const uint32_t d = tmem + g * tg;
          if (MODE == kFwd) {
            const uint32_t a = dh_k + g * gs, b = dd_k + s * ss;
#pragma unroll
            for (int k = 0; k < 4; ++k) mma(d + 128, a + k * 2, b + k * 2, id_y, add || k > 0);
          } else if (MODE == kDx) {
            const uint32_t a = dh_k + g * gs, b = dw_mn + s * ss;
#pragma unroll
            for (int k = 0; k < WR / 16; ++k)
              mma(d + 192, a + (k >> 2) * kBlk + (k & 3) * 2, b + k * 128, id_dx, add || k > 0);
          } else {
            const uint32_t a = dh_mn + g * gs, b = dx_mn + g * gs;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma(acc_gu, a + k * 128, b + k * 128, id_wx, begun || k > 0);
            const uint32_t ad = a + (GATED ? kBlk : 0), bd = dy_mn + g * gs;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma(acc_d, ad + k * 128, bd + k * 128, id_wy, begun || k > 0);
          }
          if (last_chunk) commit(out_done(g));
          if (ring) commit(empty(s));
          if (last) commit(all_done);
        }
        __syncwarp();
      };
      // Each group goes through: first product (its rows and the chunk's weights are there), hidden
      // operand ready, second product. The groups are served in the order they become ready.
      const bool ring = nch > p.nst;
      struct State {
        int left, c, s;    // chunks to go, chunk, weight stage
        uint32_t ph;       // bit 0 weights, bit 1 hidden operand, bit 2 rows
        bool fresh;        // the stage's weights are to be waited for
        bool first;        // the first product is next
        bool rows;         // ... of a new tile
      };
      State st[kMaxGroups];
      int left = p.ng * nt * nch;
#pragma unroll
      for (int g = 0; g < kMaxGroups; ++g) st[g] = {g < p.ng ? nt * nch : 0, 0, 0, 0u, true, true, true};
      bool begun = false;
      int turn = 0;  // weights: both groups add to one accumulator, always in the same order
      long long since = clock64();
      auto is_there = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try(bar, parity)) || *failed;
      };
      while (left > 0) {
        bool moved = false;
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g) {
          State& t = st[g];
          if (t.left == 0) continue;
          if (t.first) {
            if (t.fresh && !is_there(full(t.s), t.ph & 1)) continue;
            if (t.rows && !is_there(x_ready(g), (t.ph >> 2) & 1)) continue;
            fence_after();
            if (t.rows) t.ph ^= 4;
            t.rows = false;
            first_product(g, t.s);
            t.first = false;
            moved = true;
          } else if ((MODE != kDw || g == turn) && is_there(h_ready(g), (t.ph >> 1) & 1)) {
            fence_after();
            t.ph ^= 2;
            const bool last_chunk = t.c == nch - 1;
            --left;
            --t.left;
            if (p.ng > 1) turn ^= 1;
            second_product(g, t.s, t.c > 0, begun, last_chunk, ring, left == 0);
            begun = true;
            t.c = last_chunk ? 0 : t.c + 1;
            if (++t.s == p.nst) {
              t.s = 0;
              t.ph ^= 1;
              t.fresh = ring;
            }
            t.first = true;
            t.rows = last_chunk;
            moved = true;
            // within a tile the next first product follows at once when its weights are there
            if (t.left > 0 && !t.rows && (!t.fresh || is_there(full(t.s), t.ph & 1))) {
              fence_after();
              first_product(g, t.s);
              t.first = false;
            }
          }
        }
        if (moved) {
          since = clock64();
        } else if (clock64() - since > kWaitClocks) {
          *failed = 1;
          atomicOr(status, 1u);
        }
      }
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
      auto prefetch = [&](int n) {
        if (n >= nt) return;
        const long long r = (first + g + n * step) * kTile + (tid & (kTile - 1));
        if (tid < kTile)
          prefetch_row(p.x, r, p.f.M);
        else if (MODE != kFwd)
          prefetch_row(p.dy, r, p.f.M);
      };
      auto arrive = [&](uint32_t bar) {
        fence_async_shared();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      auto group_sync = [&]() {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(kGroupThreads) : "memory");
      };
      // the rows of step n; in weights mode the tile's old rows are free once out_done came
      uint32_t ph_gu = 0, ph_out = 0;
      auto wait_out = [&]() {
        mbar_wait(out_done(g), ph_out, failed, status);
        ph_out ^= 1;
        fence_after();
      };
      auto load = [&](int n, bool wait) {
        const long long r0 = (first + g + n * step) * kTile;
        uint4 bx[4], by[4];
        if (p.x.aligned) fetch_rows(p.x, 0, r0, p.f.M, tid, bx);
        if (MODE != kFwd && p.dy.aligned) fetch_rows(p.dy, 0, r0, p.f.M, tid, by);
        if (wait) wait_out();
        auto rest = [&](const RowSrc& src, int blocks, uint4 (&v)[4], uint8_t* dst) {
          if (src.aligned) {
            store_rows(0, tid, v, dst);
            if (blocks > 1) {
              fetch_rows(src, 1, r0, p.f.M, tid, v);
              store_rows(1, tid, v, dst);
            }
          } else {
            for (int b = 0; b < blocks; ++b) gather_rows(src, b, r0, p.f.M, tid, dst);
          }
        };
        rest(p.x, nbx, bx, Xs);
        if (MODE != kFwd) rest(p.dy, nby, by, Ys);
        arrive(x_ready(g));
      };
      // this thread: row `row` of the tile, units half * 32 .. + 32, taken kUnits at a time; the
      // next units' accumulators are on their way while one set is worked on
      constexpr int kUnits = MODE == kFwd ? 16 : 8;
      constexpr int kSteps = 32 / kUnits;
      auto get = [&](int q, uint32_t (&ra)[kUnits], uint32_t (&ru)[kUnits],
                     uint32_t (&rd)[kUnits]) {
        const uint32_t at = d + half * 32 + q * kUnits;
        tmem_ld(at, ra);
        if (GATED) tmem_ld(at + 64, ru);
        if (MODE != kFwd) tmem_ld(at + 128, rd);
      };
      auto work = [&](int q, const uint32_t (&ra)[kUnits], const uint32_t (&ru)[kUnits],
                      const uint32_t (&rd)[kUnits]) {
        uint32_t h[kUnits / 2], da[kUnits / 2], du[kUnits / 2];
#pragma unroll
        for (int e = 0; e < kUnits; e += 4) {
          float a[4], f[4], sl[4], vh[4], va[4], vu[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = __uint_as_float(ra[e + i]);
          act4<ACT, MODE != kFwd>(a, f, sl);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = GATED ? __uint_as_float(ru[e + i]) : 1.0f;
            vh[i] = GATED ? f[i] * u : f[i];
            if (MODE != kFwd) {
              const float dh = __uint_as_float(rd[e + i]);
              va[i] = GATED ? dh * u * sl[i] : dh * sl[i];
              vu[i] = dh * f[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            h[(e + i) / 2] = Two<T>::pack(vh[i], vh[i + 1]);
            if (MODE != kFwd) {
              da[(e + i) / 2] = Two<T>::pack(va[i], va[i + 1]);
              du[(e + i) / 2] = Two<T>::pack(vu[i], vu[i + 1]);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < kUnits; e += 8) {
          const int piece = half * 4 + (q * kUnits + e) / 8;
          uint8_t* at = Hs + row * 128 + ((piece ^ (row & 7)) << 4);
          auto put = [&](int block, const uint32_t* v) {
            *reinterpret_cast<uint4*>(at + block * 16384) = make_uint4(v[0], v[1], v[2], v[3]);
          };
          if (MODE == kFwd) {
            put(0, h + e / 2);
          } else {
            put(0, da + e / 2);
            if (GATED) put(1, du + e / 2);
            if (MODE == kDw) put(GATED ? 2 : 1, h + e / 2);
          }
        }
      };
      auto landed = [&](uint32_t (&ra)[kUnits], uint32_t (&ru)[kUnits], uint32_t (&rd)[kUnits]) {
        tmem_wait(ra);
        if (GATED) tmem_wait(ru);
        if (MODE != kFwd) tmem_wait(rd);
      };

      prefetch(1);
      load(0, false);
      for (int n = 0; n < nt; ++n) {
        prefetch(n + 2);
        for (int c = 0; c < nch; ++c) {
          mbar_wait(gu_full(g), ph_gu, failed, status);
          ph_gu ^= 1;
          fence_after();
          uint32_t a0[kUnits], u0[kUnits], d0[kUnits], a1[kUnits], u1[kUnits], d1[kUnits];
          get(0, a0, u0, d0);
#pragma unroll
          for (int q = 0; q < kSteps; q += 2) {
            landed(a0, u0, d0);
            get(q + 1, a1, u1, d1);
            work(q, a0, u0, d0);
            landed(a1, u1, d1);
            if (q + 2 < kSteps) get(q + 2, a0, u0, d0);
            work(q + 1, a1, u1, d1);
          }
          arrive(h_ready(g));
        }
        // the tile's first products are done, so its rows make room for the next tile's (weights:
        // after the second product, which reads them too)
        const bool more = n + 1 < nt;
        if (more) load(n + 1, MODE == kDw);
        if (MODE != kDw) {
          wait_out();
          // results to shared memory (the hidden operand's place, free now), then out
          const int cols = MODE == kFwd ? p.f.O : p.f.D;
          const uint32_t src = d + (MODE == kFwd ? 128 : 192) + half * 32;
          for (int b = 0; b * 64 < cols; ++b) {
            if (b * 64 + half * 32 < cols) {
              uint32_t v0[16], v1[16];
              tmem_ld(src + b * 64, v0);
              tmem_ld(src + b * 64 + 16, v1);  // (inside the accumulator's 32-column padding)
              tmem_wait(v0);
              tmem_wait(v1);
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                  const int i = (e + k) & 15;
                  w[k / 2] = e < 16 ? Two<T>::pack(__uint_as_float(v0[i]), __uint_as_float(v0[i + 1]))
                                    : Two<T>::pack(__uint_as_float(v1[i]), __uint_as_float(v1[i + 1]));
                }
                *reinterpret_cast<uint4*>(Hs + row * 128 +
                                          (((half * 4 + e / 8) ^ (row & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
            group_sync();
            write_rows(Hs, (uint8_t*)(MODE == kFwd ? p.f.y : p.f.dx),
                       2 * (MODE == kFwd ? p.f.ldy : p.f.lddx), p.out_aligned, b * 64, cols,
                       (first + g + n * step) * kTile, p.f.M, tid);
            group_sync();
          }
        } else if (!more) {
          wait_out();
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
        tmem_ld((which ? acc_d : acc_gu) + row_lanes + e0, v);
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

bool aligned16(const void* p, long long ld, int cols) {
  return (((uintptr_t)p | (uintptr_t)(ld * 2) | (uintptr_t)(cols * 2)) & 15) == 0;
}

RowSrc row_src(const void* p, long long ld, long long rows, int cols) {
  RowSrc s = {};
  if (rows <= 0) return s;
  s.base = (const uint8_t*)p;
  s.ld = rows > 1 ? ld * 2 : 0;
  s.cols = cols;
  s.aligned = aligned16(p, s.ld / 2, cols);
  s.lo = (const uint8_t*)(((uintptr_t)p + 15) & ~(uintptr_t)15);
  s.hi = (const uint8_t*)(((uintptr_t)p + (uintptr_t)((rows - 1) * ld * 2 + cols * 2)) &
                          ~(uintptr_t)15);
  return s;
}

int pad16(int v) { return (v + 15) & ~15; }

int stage_bytes(int D, int O, bool gated) {
  return (D + 63) / 64 * (gated ? 128 : 64) * 128 + pad16(O) * 128;
}

template <int MODE, typename T, int ACT, bool GATED>
int launch(TcArgs p, cudaStream_t st) {
  const bool one = p.f.M <= 1;  // a single row's stride is never used
  p.x = row_src(p.f.x, p.f.ldx, p.f.M, p.f.D);
  if (MODE != kFwd) p.dy = row_src(p.f.dy, p.f.lddy, p.f.M, p.f.O);
  if (MODE == kFwd) p.out_aligned = aligned16(p.f.y, one ? 0 : p.f.ldy, p.f.O);
  if (MODE == kDx) p.out_aligned = aligned16(p.f.dx, one ? 0 : p.f.lddx, p.f.D);
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

cudaError_t ffn_status_take(unsigned int* out, cudaStream_t st) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_rows_status, sizeof *out, 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_rows_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
  return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

}  // namespace rows
}  // namespace splat
