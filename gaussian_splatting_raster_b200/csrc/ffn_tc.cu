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
// A CTA's work is one sequence of items, (tile, chunk) or tiles. Two groups of eight warps turn
// accumulators into hidden values, item by item in turn; one warp issues the first products, up to
// three items ahead, and loads weights; one warp issues the second products of the items that are
// ready; two warps bring row tiles in. So the tensor cores and the groups wait for one another only
// at the ends of the sequence: what bounds a narrow block is the groups' arithmetic (special
// function unit and issue slots), a wide one the tensor cores and L2. (With an accumulator per
// group, a group waited about as long for its products as it worked on them.) Weights are packed
// once per call into the layout the MMAs read (zeros beyond F, D and O), so a chunk is one
// contiguous bulk copy; all chunks stay in shared memory where they fit. Row tiles come through a
// tensor map where rows are 16-byte aligned; else (token rows have odd widths) as one bulk copy of
// the bytes a tile spans, which the loaders lay out from shared memory; at the array's ends,
// element by element.
//
// Measured, bf16, silu, gated, the kernel by itself: forward, 917,504 rows of 64 / 256 / 64 187 us
// (482 TFLOP/s of products; issue slots 57 %, special function unit 48 %, tensor pipe 23 %; without
// a gate 175 us), 200,000 rows of 128 / 512 / 128 127 us (617 TFLOP/s). Gradients, 311,296 rows of
// 64 / 128 / 64: dx 51 us, weights 63; of 35 / 128 / 48 in rows 76 bytes apart, where the loaders
// bound it, 116 and 115. Few tiles (1,000 rows of 57 / 256 / 64, nothing in L2) take 9 us, dx 20,
// weights 17.
#include <cuda.h>

#include <algorithm>

#include "ffn.cuh"
#include "tc.cuh"

namespace splat {
namespace rows {
namespace {

using namespace tc;

enum Mode { kFwd, kDx, kDw };

constexpr int kGroupThreads = 256;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kLoaders = 64;
constexpr int kTcThreads = 2 * kGroupThreads + 64 + kLoaders;  // + both products, + row tiles
constexpr int kMaxStages = 16;
constexpr int kMaxGu = 3, kMaxRows = 3;  // accumulators of first products; row tiles
constexpr int kTile = 128;
// Rows whose weight gradients one accumulator takes: a launch has at most so many a split, and adds
// its sums to those of the launch before. The tensor cores add with truncation: a sum of one sign
// loses up to 2^-22 of what it holds with every 16 rows (measured: 0.82 of that), so 5e-5 of itself
// over 8,192 rows and 4e-4 over 65,536, a tenth of the type's rounding; over 131,072 it was 8e-4 in
// fp16 too. Each launch more costs about 12 us: 917,504 rows of 64 / 256 / 64 take 280 us in bf16,
// which is one, and 320 in fp16, which is four.
constexpr long long sum_rows(bool bf16) { return bf16 ? 65536 : 8192; }
constexpr int kSmemLimit = 232448 - 2048;  // 227 KB less the alignment slack and the barriers

__device__ unsigned int g_rows_status;

// A row array as the loads see it: words may be taken from [lo, hi) only.
struct RowSrc {
  const uint8_t *base, *lo, *hi;  // lo, hi: 4-byte aligned, inside the array
  long long ld;                   // bytes
  int cols, tiled;                // tiled: read through the tensor map
  int raw;                        // else bytes of a tile as it lies in memory, 0: not staged
};

// Narrow blocks take 32 hidden units a chunk, and its other 32 places hold the same units again,
// whose hidden values and gradients are stored as what rounding took from the first ones: the
// second products then have them in twice the bits. With at most 32 hidden units that is free;
// otherwise it costs the groups' work twice (758,527 rows of 2 / 104 / 21: 239 us instead of 120).
// Sums over few units, or over units that are functions of few inputs, have little to average the
// roundings: the weight gradients of one unit were off by several times their own rounding, outputs
// of two inputs by 1.5 times. (About D^2 / 4 products of inputs in O outputs are independent.) In
// other blocks the one rounding stays: it brings outputs from 0.17 % off (their own rounding, in
// bf16) to 0.24 %, and twice the bits would cost twice the groups' work there.
__host__ __device__ constexpr bool twice(int D, int F, int O) { return F <= 32 || D * D * O < 512; }
// units of a chunk
__host__ __device__ constexpr int units(int D, int F, int O) {
  return twice(D, F, O) ? 32 : kChunk;
}

struct TcArgs {
  FfnArgs f;
  const uint8_t* img;   // packed weights, chunk after chunk
  int nch, stage_bytes; // chunks; bytes of one
  int units;            // hidden units of a chunk: 64, or 32 that are there twice
  int nst, nx, nh;      // weight stages, row tiles and hidden operands in shared memory
  int ngu, no;          // accumulators of first products and of outputs in TMEM
  int staged;           // outputs have places of their own in shared memory
  int raw_off;          // where tiles lie as in memory (x, then dy)
  int dp, op;           // D and O rounded up to 16
  RowSrc x, dy;
  int out_aligned;      // y's or dx's rows start and end at 16 bytes
  int out_dense;        // ... lie one behind the other from a 16-byte boundary
  long long tiles;
  int again;            // weight gradients: the CTAs' sums are added to
  int pack_ctas;        // CTAs of the packing kernel that pack; those behind them look at dy
  int parts;            // ... their number, 0 but in fp16 gradients
};

// a - r, nothing where the rounded r is infinite or no number
__device__ __forceinline__ float left(float a, float r) {
  return fabsf(r) < __int_as_float(0x7f800000) ? a - r : 0.0f;
}

// pairs in the type: rounded, and what the rounding left (also rounded)
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint32_t rest(float a, float b) {
    return pack(left(a, __bfloat162float(__float2bfloat16_rn(a))),
                left(b, __bfloat162float(__float2bfloat16_rn(b))));
  }
};
template <> struct Two<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint32_t rest(float a, float b) {
    return pack(left(a, __half2float(__float2half_rn(a))), left(b, __half2float(__float2half_rn(b))));
  }
};

// two fp32 lanes of one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Four reciprocals are taken as one, since the special function unit takes one value per lane group
// and cycle (16 an SM), which is what bounds these kernels at narrow widths: with
// r = 1 / (p0 p1 p2 p3) each is r times the product of the other three. False
// where the product is out of range or no number: the four mean nothing then.
__device__ __forceinline__ bool rcp4(const float2 (&p)[2], float2 (&r)[2]) {
  const float2 m = mul2(p[0], p[1]);  // p0 p2, p1 p3
  const float all = m.x * m.y;
  const float i = rcp_fast(all);
  const float2 w = make_float2(i * m.y, i * m.x);
  r[0] = mul2(w, p[1]);
  r[1] = mul2(w, p[0]);
  return all < 4.253529586511731e37f;  // 2^125
}

// act and its slope for four values (without SLOPE the slope is not formed).
//   silu: s = 1 / (1 + 2^t), t = -a log2 e. Where the four factors' product leaves the range (some a
//         are far on the left, or no number) the result is false and f and slope mean nothing; then
//         ALONE: a reciprocal for each value, zero once 2^t is infinite, so that a s goes to zero with
//         s. (That way for all values would take two results of the special function unit a value.)
//   gelu: Phi by Abramowitz and Stegun 7.1.26 (erfc at z = |a| / sqrt 2, absolute error 0.75e-7 in
//         Phi; relative error of Phi(-|a|) 0.05 % at -4, 0.8 % at -7.5), z held at 10 where
//         Phi(-|a|) has long become zero; one power e^{-a^2/2} serves Phi and the density.
// An argument that is no number gives no number: both are multiplied by a, or built from it.
constexpr float kFar = -21.0f;  // four values from here on keep the product below 2^122

__device__ __forceinline__ float min_nan(float a, float b) {  // no number if one of them is none
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int ACT, bool SLOPE, bool ALONE>
__device__ __forceinline__ bool act4(const float2 (&a)[2], float2 (&f)[2], float2 (&slope)[2]) {
  float2 p[2], r[2];
  bool ok = true;
  if (ACT == SPLAT_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 t = mul2(a[i], both(-1.4426950408889634f));
      p[i] = add2(make_float2(ex2_fast(t.x), ex2_fast(t.y)), both(1.0f));
    }
    if (ALONE) {
#pragma unroll
      for (int i = 0; i < 2; ++i) r[i] = make_float2(rcp_fast(p[i].x), rcp_fast(p[i].y));
    } else {
      ok = rcp4(p, r);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[i] = mul2(a[i], r[i]);
      if (SLOPE) slope[i] = fma2(f[i], fma2(r[i], both(-1.0f), both(1.0f)), r[i]);
    }
  } else {
    float2 z[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      z[i] = mul2(a[i], both(0.70710678118654752f));
      z[i] = make_float2(fminf(fabsf(z[i].x), 10.0f), fminf(fabsf(z[i].y), 10.0f));
      p[i] = fma2(both(0.3275911f), z[i], both(1.0f));
    }
    rcp4(p, r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 t = mul2(mul2(z[i], z[i]), both(-1.4426950408889634f));
      const float2 e = make_float2(ex2_fast(t.x), ex2_fast(t.y));
      // half the published coefficients
      float2 q = fma2(both(0.5307027145f), r[i], both(-0.7265760135f));
      q = fma2(q, r[i], both(0.7107068705f));
      q = fma2(q, r[i], both(-0.142248368f));
      q = fma2(q, r[i], both(0.127414796f));
      q = mul2(mul2(q, r[i]), e);
      const float2 c = make_float2(a[i].x >= 0.0f ? 1.0f - q.x : q.x,
                                   a[i].y >= 0.0f ? 1.0f - q.y : q.y);
      f[i] = mul2(a[i], c);
      if (SLOPE) slope[i] = fma2(mul2(a[i], both(0.3989422804014327f)), e, c);
    }
  }
  return ok;
}

// ---------------------------------------------------------------------------------------------
// packed weights
// ---------------------------------------------------------------------------------------------
// In fp16 the gradients of hidden values, da and du, are held times a power of two: gradients of a
// mean over many rows are near fp16's smallest step (6e-8) and below it they would be zero, large
// ones infinite. The power is 1 while the largest finite |dy| is in [2^-6, 16), else it brings it
// into [2^-6, 2^-5) or [1, 2): da and du keep fp16's digits down to 2^-8 of the largest |dy| and
// may grow to 2^11 times it (small |dy|: 2^21, large: 2^15). Sums are fp32 and are scaled back,
// exactly. It costs one pass over dy, along with the packing of the weights, and a product a hidden
// value: gradients of 311,296 rows of 35 / 128 / 48 take 12 us and 5 % more than in bf16.
__device__ __forceinline__ int hidden_shift(unsigned max_bits) {  // fp16 bits, without a sign
  const float m = __half2float(__ushort_as_half((unsigned short)max_bits));
  const int e = ((__float_as_int(m) >> 23) & 255) - 127;  // (subnormal fp16 values are normal here)
  return max_bits == 0 ? 0 : e < -6 ? -6 - e : e >= 4 ? -e : 0;
}
__device__ __forceinline__ float power_of_two(int k) { return __int_as_float((127 + k) << 23); }

// The largest finite |dy| of rows part, part + parts, ... by 16 a warp: lanes have the words of a
// row (every 32nd of H), and the elements before the first and behind the last word of a row each.
template <int H>
__device__ __forceinline__ unsigned dy_rows(const FfnArgs& f, int part, int parts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int U = 16;
  const uint16_t* dy = (const uint16_t*)f.dy;
  unsigned m = 0;
  auto take = [&](uint32_t w) {
    const unsigned lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
    if (lo < 0x7C00u) m = max(m, lo);
    if (hi < 0x7C00u) m = max(m, hi);
  };
  for (long long r0 = (part * 8LL + warp) * U; r0 < f.M; r0 += (long long)parts * 8 * U) {
    const int n = (int)min((long long)U, f.M - r0);
    const uint16_t* row = dy + r0 * f.lddy;
    uint32_t w[H][U], ends = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint16_t* q = row + u * f.lddy;
      const int odd = ((uintptr_t)q & 2) >> 1;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int c = 2 * (lane + 32 * h) + odd;
        w[h][u] = 0u;
        if (u < n && c + 1 < f.O) w[h][u] = __ldg(reinterpret_cast<const uint32_t*>(q + c));
      }
    }
    if (lane < n) {
      const uint16_t* q = row + lane * f.lddy;
      const int odd = ((uintptr_t)q & 2) >> 1;
      if (odd) ends = __ldg(q);
      if ((f.O - odd) & 1) ends |= (uint32_t)__ldg(q + f.O - 1) << 16;
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int u = 0; u < U; ++u) take(w[h][u]);
    take(ends);
  }
  return m;
}

__device__ __forceinline__ void dy_part(const FfnArgs& f, int part, int parts) {
  __shared__ unsigned s_max;
  if (threadIdx.x == 0) s_max = 0;
  __syncthreads();
  unsigned m = f.O <= 64 ? dy_rows<1>(f, part, parts) : dy_rows<2>(f, part, parts);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_max, m);
  __syncthreads();
  if (threadIdx.x == 0) f.dy_max[part] = s_max;
}

// Chunk c: [Wg units | Wu units] (128 rows, 64 without a gate) in blocks of 64 columns of D, then
// Wd's columns of the chunk (op rows of 64). One thread per 16-byte piece.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256)
k_pack(TcArgs p, uint8_t* __restrict__ img) {
  if (!Two<T>::kBf16 && (int)blockIdx.x >= p.pack_ctas) {
    dy_part(p.f, blockIdx.x - p.pack_ctas, p.parts);
    return;
  }
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
    const int f = c * p.units + (row & (p.units - 1));
    if (f < p.f.F) {
      src = (const T*)(GATED && row < 64 ? p.f.wg : p.f.wu) + (size_t)f * p.f.D + col;
      n = p.f.D - col;
    }
  } else {
    row = (q - gu) >> 3;
    const int unit = (((q - gu) & 7) ^ (row & 7)) << 3;
    const int col = c * p.units + (unit & (p.units - 1));
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

// Row tiles come by TMA where the rows allow it (start and distance multiples of 16 bytes): one
// instruction a 64-column block, zeros behind the last row and column. Any other rows (odd widths
// start anywhere) come as they lie in memory, gaps between rows included, by one bulk copy into
// shared memory, from where the loader warps put them into place; where there is no room for that,
// and at the array's ends where a copy's 16 bytes would reach over them, the loader warps read the
// rows from global memory.
//
// Eight threads to a row: thread t has piece t & 7 (8 elements) of the block in rows t / 8 + 8 j,
// read as the five words around it and shifted by half a word where the row starts on an odd
// element. Rows >= M are zeros, and so are elements behind a row's end up to the block's.
struct Piece {
  uint32_t w[5];
};

// words to the piece's place: `keep` has the bits of its elements
__device__ __forceinline__ void put_piece(uint8_t* q, const Piece& v, uint32_t sh,
                                          const uint4& keep) {
  *reinterpret_cast<uint4*>(q) =
      make_uint4(__funnelshift_r(v.w[0], v.w[1], sh) & keep.x,
                 __funnelshift_r(v.w[1], v.w[2], sh) & keep.y,
                 __funnelshift_r(v.w[2], v.w[3], sh) & keep.z,
                 __funnelshift_r(v.w[3], v.w[4], sh) & keep.w);
}

__device__ __forceinline__ uint4 keep_bits(int n) {  // of the first n of 8 elements
  uint32_t m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    m[k] = n >= 2 * k + 2 ? 0xFFFFFFFFu : n == 2 * k + 1 ? 0xFFFFu : 0u;
  return make_uint4(m[0], m[1], m[2], m[3]);
}

// from the staged tile at `at` (whose buffer has room for the words behind its last row)
__device__ __forceinline__ void place_staged(uint32_t at, int ld, int cols, int block,
                                             long long rows, int tid, uint8_t* dst) {
  const int c = block * 8 + (tid & 7), r = tid >> 3;
  const uint4 keep = keep_bits(cols - c * 8), none = make_uint4(0u, 0u, 0u, 0u);
  // (pieces behind the row's end read what is there, within the buffer, and keep nothing)
  uint32_t p = at + r * ld + (c * 8 < cols ? c * 16 : 0);
  uint8_t* q = dst + block * 16384 + r * 128 + (((tid & 7) ^ (r & 7)) << 4);
  constexpr int U = 8;
#pragma unroll
  for (int j0 = 0; j0 < kTile / 8; j0 += U) {
    Piece v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t a = (p + j * 8 * ld) & ~3u;
#pragma unroll
      for (int k = 0; k < 5; ++k)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[j].w[k]) : "r"(a + 4 * k));
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
      put_piece(q + (j0 + j) * 1024, v[j], ((p + j * 8 * ld) & 2u) * 8u,
                r + 8 * (j0 + j) < rows ? keep : none);
    p += 8 * U * ld;
  }
}

// from global memory; at the array's ends element by element
__device__ __forceinline__ void place_rows(const RowSrc& s, long long r0, int block,
                                           long long rows, int tid, uint8_t* dst) {
  const int c = block * 8 + (tid & 7), r = tid >> 3;
  const int n = min(8, s.cols - c * 8);  // elements wanted
  const uint4 keep = keep_bits(n);
  const uint8_t* p = s.base + (r0 + r) * s.ld + c * 16;
  uint8_t* q = dst + block * 16384 + r * 128 + (((tid & 7) ^ (r & 7)) << 4);
  constexpr int U = 4;
#pragma unroll 1
  for (int j0 = 0; j0 < kTile / 8; j0 += U, p += 8 * U * s.ld, q += U * 1024) {
    Piece v[U];
    uint32_t sh[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint8_t* e = p + 8 * j * s.ld;
      const uint8_t* a = (const uint8_t*)((uintptr_t)e & ~(uintptr_t)3);
      sh[j] = ((uint32_t)(uintptr_t)e & 2u) * 8u;
      const int words = n > 0 && r + 8 * (j0 + j) < rows ? (2 * n + (int)(sh[j] >> 3) + 3) >> 2 : 0;
      const bool whole = a >= s.lo && a + 4 * words <= s.hi;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        v[j].w[k] = 0u;
        if (k < words) {
          if (whole) {
            v[j].w[k] = __ldg(reinterpret_cast<const uint32_t*>(a) + k);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint8_t* x = a + 4 * k + 2 * h;
              if (x >= e && x < e + 2 * n)
                v[j].w[k] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(x)) << (16 * h);
            }
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) put_piece(q + j * 1024, v[j], sh[j], keep);
  }
}

// The bulk copy of the tile at row r0: start and bytes, 0 when it would reach over the array's ends.
__device__ __forceinline__ uint32_t raw_span(const RowSrc& s, long long r0, long long M,
                                             const uint8_t*& start) {
  const uint8_t* p = s.base + r0 * s.ld;
  start = (const uint8_t*)((uintptr_t)p & ~(uintptr_t)15);
  const long long rows = min((long long)kTile, M - r0);
  const long long last = (long long)(p - start) + (rows - 1) * s.ld + s.cols * 2;
  const long long bytes = (last + 15) & ~15LL;
  if (start < s.lo || start + bytes > s.hi) return 0;
  return (uint32_t)bytes;
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

// TMEM columns of a first product: A|U (A), and dH behind it in the gradients
__host__ __device__ constexpr int gu_cols(int mode, bool gated) {
  return (gated ? 128 : 64) + (mode == kFwd ? 0 : 64);
}
__host__ __device__ constexpr int pad32(int v) { return (v + 31) & ~31; }

// shared memory of a row tile, and of a hidden operand (h; da, du; da, du, h)
__host__ __device__ constexpr int rows_bytes(int mode, int dp, int op) {
  return ((dp + 63) / 64 + (mode == kFwd ? 0 : (op + 63) / 64)) * 16384;
}
__host__ __device__ constexpr int hidden_bytes(int mode, bool gated) {
  return (mode == kFwd ? 1 : (gated ? 2 : 1) + (mode == kDw ? 1 : 0)) * 16384;
}

// values of a row's hidden operand in the type: rounded, or what rounding took from them
template <typename T, bool AGAIN>
__device__ __forceinline__ uint32_t held(float a, float b) {
  return AGAIN ? Two<T>::rest(a, b) : Two<T>::pack(a, b);
}

// Units of a row: accumulators (a, u, dh) to values of the hidden operand, as pairs; false where
// some four units have to be taken ALONE.
template <int MODE, typename T, int ACT, bool GATED, bool AGAIN, bool ALONE, int kUnits>
__device__ __forceinline__ bool hidden_values(const uint32_t (&ra)[kUnits],
                                              const uint32_t (&ru)[kUnits],
                                              const uint32_t (&rd)[kUnits], float scale,
                                              uint32_t (&h)[kUnits / 2],
                                              uint32_t (&da)[kUnits / 2],
                                              uint32_t (&du)[kUnits / 2]) {
  bool ok = true;
#pragma unroll
  for (int e = 0; e < kUnits; e += 4) {
    auto two = [&](const uint32_t (&r)[kUnits], int k) {
      return make_float2(__uint_as_float(r[e + 2 * k]), __uint_as_float(r[e + 2 * k + 1]));
    };
    const float2 a[2] = {two(ra, 0), two(ra, 1)};
    float2 f[2], sl[2];
    ok &= act4<ACT, MODE != kFwd, ALONE>(a, f, sl);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float2 u = make_float2(1.0f, 1.0f);
      if (GATED) u = two(ru, k);
      if (MODE != kDx) {
        const float2 v = GATED ? mul2(f[k], u) : f[k];
        h[e / 2 + k] = held<T, AGAIN>(v.x, v.y);
      }
      if (MODE != kFwd) {
        const float2 dh = Two<T>::kBf16 ? two(rd, k) : mul2(two(rd, k), both(scale));
        const float2 va = mul2(GATED ? mul2(dh, u) : dh, sl[k]);
        da[e / 2 + k] = held<T, AGAIN>(va.x, va.y);
        if (GATED) {
          const float2 vu = mul2(dh, f[k]);
          du[e / 2 + k] = held<T, AGAIN>(vu.x, vu.y);
        }
      }
    }
  }
  return ok;
}

// the operand's blocks: put(block, its pairs)
template <int MODE, bool GATED, typename F>
__device__ __forceinline__ void hidden_blocks(const uint32_t* h, const uint32_t* da,
                                              const uint32_t* du, F put) {
  if (MODE == kFwd) {
    put(0, h);
  } else {
    put(0, da);
    if (GATED) put(1, du);
    if (MODE == kDw) put(GATED ? 2 : 1, h);
  }
}

// ... into the operand's 16-byte pieces piece ..
template <int MODE, typename T, int ACT, bool GATED, bool AGAIN, int kUnits>
__device__ __forceinline__ bool hidden_units(uint8_t* Hs, int row, int piece,
                                             const uint32_t (&ra)[kUnits],
                                             const uint32_t (&ru)[kUnits],
                                             const uint32_t (&rd)[kUnits], float scale) {
  uint32_t h[kUnits / 2], da[kUnits / 2], du[kUnits / 2];
  const bool ok =
      hidden_values<MODE, T, ACT, GATED, AGAIN, false, kUnits>(ra, ru, rd, scale, h, da, du);
#pragma unroll
  for (int e = 0; e < kUnits; e += 8) {
    uint8_t* at = Hs + row * 128 + (((piece + e / 8) ^ (row & 7)) << 4);
    hidden_blocks<MODE, GATED>(h + e / 2, da + e / 2, du + e / 2, [&](int block, const uint32_t* v) {
      *reinterpret_cast<uint4*>(at + block * 16384) = make_uint4(v[0], v[1], v[2], v[3]);
    });
  }
  return ok;
}

// four units ALONE, into half a piece, for the lanes that want them
template <int MODE, typename T, int ACT, bool GATED, bool AGAIN>
__device__ __forceinline__ void hidden_alone(uint8_t* at, bool want, const uint32_t (&ra)[4],
                                             const uint32_t (&ru)[4], const uint32_t (&rd)[4],
                                             float scale) {
  uint32_t h[2], da[2], du[2];
  hidden_values<MODE, T, ACT, GATED, AGAIN, true, 4>(ra, ru, rd, scale, h, da, du);
  if (want)
    hidden_blocks<MODE, GATED>(h, da, du, [&](int block, const uint32_t* v) {
      *reinterpret_cast<uint2*>(at + block * 16384) = make_uint2(v[0], v[1]);
    });
}

template <int MODE, typename T, int ACT, bool GATED, bool TWICE>
__global__ void __launch_bounds__(kTcThreads, 1)
k_ffn_tc(const __grid_constant__ TcArgs p, const __grid_constant__ CUtensorMap x_map,
         const __grid_constant__ CUtensorMap dy_map) {
  extern __shared__ uint8_t raw[];
  constexpr int kBars = 2 * kMaxStages + 2 * kMaxGu + 2 * kMaxRows + 2 + 2 + 2 + 2 + 2;
  __shared__ __align__(8) uint64_t s_bar[kBars];
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  constexpr int WR = GATED ? 128 : 64;
  constexpr bool BF = Two<T>::kBf16;
  constexpr uint32_t kGu = gu_cols(MODE, GATED);
  constexpr uint32_t kHBytes = hidden_bytes(MODE, GATED);
  constexpr bool kScaled = !BF && MODE != kFwd;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int shift = 0;
  if (kScaled && warp < 2 * kGroupWarps) {
    unsigned m = 0;
    for (int i = lane; i < p.parts; i += 32) m = max(m, __ldg(p.f.dy_max + i));
    shift = hidden_shift(__reduce_max_sync(0xffffffffu, m));
  }
  const float back = power_of_two(-shift);
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int nbx = (p.dp + 63) >> 6, nby = (p.op + 63) >> 6;
  const uint32_t xbytes = rows_bytes(MODE, p.dp, p.op);
  const uint32_t x_off = p.nst * p.stage_bytes, h_off = x_off + p.nx * xbytes;
  const uint32_t bars = smem_addr(s_bar);
  auto full = [&](int k) { return bars + 8 * k; };                    // a stage's weights are there
  auto empty = [&](int k) { return bars + 8 * (kMaxStages + k); };    // ... are used
  constexpr int kB0 = 2 * kMaxStages;
  auto gu_full = [&](int k) { return bars + 8 * (kB0 + k); };         // a first product is done
  auto gu_free = [&](int k) { return bars + 8 * (kB0 + kMaxGu + k); };  // ... has been read
  constexpr int kB2 = kB0 + 2 * kMaxGu;
  auto x_ready = [&](int k) { return bars + 8 * (kB2 + k); };           // a row tile is there
  auto x_free = [&](int k) { return bars + 8 * (kB2 + kMaxRows + k); };  // ... is used
  constexpr int kB1 = kB2 + 2 * kMaxRows;
  auto h_ready = [&](int k) { return bars + 8 * (kB1 + k); };     // item's hidden operand, by parity
  auto done = [&](int k) { return bars + 8 * (kB1 + 2 + k); };    // item's second product, by parity
  auto out_full = [&](int k) { return bars + 8 * (kB1 + 4 + k); };  // a tile's output is complete
  auto out_free = [&](int k) { return bars + 8 * (kB1 + 6 + k); };  // ... has been read
  const uint32_t all_done = bars + 8 * (kB1 + 8), raw_full = bars + 8 * (kB1 + 9);
  volatile int* failed = &s_failed;
  unsigned int* status = &g_rows_status;

  if (threadIdx.x == 0) {
    s_failed = 0;
    for (int k = 0; k < kBars; ++k) {
      const bool by_group = (k >= kB0 + kMaxGu && k < kB2) || k == kB1 || k == kB1 + 1 ||
                            k == kB1 + 6 || k == kB1 + 7;
      const bool by_loaders = k >= kB2 && k < kB2 + kMaxRows;
      mbar_init(bars + 8 * k, by_group ? kGroupWarps : by_loaders ? kLoaders / 32
                                                                    : k == kB1 + 8 ? 2 : 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_shared();
  }
  constexpr uint32_t kCols = 512;
  if (warp == 2 * kGroupWarps) tmem_alloc(smem_addr(&s_tmem), kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  // behind the first products: outputs (forward, dx), or [da|du]^T X and [du|h]^T dY
  const uint32_t acc = tmem + p.ngu * kGu;
  const uint32_t acc_step = MODE == kFwd ? pad32(p.op) : pad32(p.dp);

  const int chunk0 = MODE == kDw ? blockIdx.x % p.nch : 0;
  const int nch = MODE == kDw ? 1 : p.nch;
  const int ctas = MODE == kDw ? p.f.splits : gridDim.x;
  const int me = MODE == kDw ? blockIdx.x / p.nch : blockIdx.x;
  const int nt = me < p.tiles ? (int)((p.tiles - me + ctas - 1) / ctas) : 0;  // tiles me + n ctas
  const int total = nt * nch;                                                 // items
  const bool ring = nch > p.nst;
  // Barriers of first products. A wait tells a phase by its parity, so it must know that the phase
  // before is over and the one behind cannot be: with two barriers or more, item i - 2 (which the
  // waiting group has seen) or one before it has the phase before on item i's.
  const int gu_bars = max(p.ngu, 2);

  // descriptors count in 16 bytes: a step of 16 along K is 2 in a K-major tile (4 steps to a
  // 64-column block), 128 in an MN-major one; weights' blocks have WR rows
  constexpr uint32_t kBlk = 16384 >> 4, kWBlk = WR * 128 >> 4;
  constexpr uint32_t kMn = (16384 >> 4) << 16, kWMn = (WR * 128 >> 4) << 16, kK = 1u << 16;
  const uint32_t xs = xbytes >> 4, ss = p.stage_bytes >> 4;
  const uint32_t y_off = nbx * kBlk, down_off = nbx * kWBlk;
  if (warp == 2 * kGroupWarps) {
    // ------------------------------------------------------------- first products, weight loads
    if (nt > 0) {
      const int kx = p.dp >> 4, ko = p.op >> 4;
      const uint32_t id_gu = idesc(BF, WR, false, false), id_dh = idesc(BF, 64, false, true);
      const uint32_t x_k = desc_lo(sbase + x_off, 16), w_k = desc_lo(sbase, 16);
      // (this loop is the longest chain of an item: about 100 instructions, a fifth of an SM's
      // issue slots away; as a loop that asked its barriers in turn it took 1,000 cycles an item)
      // product: chunk, accumulator (and its barrier), rows, weights
      int c1 = 0, gu = 0, gb = 0, x1 = 0, s1 = 0;
      uint32_t pg = 1, px = 0, pw = 0;  // (the first round of accumulators is free)
      // the next chunk's weights: number, chunk, stage
      const int uses = ring ? total : nch;
      int j = 0, cj = 0, sj = 0, loads = 0;  // loads: those that were started
      uint32_t pe = 1;
      auto load_weights = [&]() {
        // (after a failed wait a stage's last phase may still be open: nothing more is started)
        if (!__any_sync(0xffffffffu, *failed)) {
          ++loads;
          if (elect_one()) {
            mbar_expect(full(sj), p.stage_bytes);
            bulk_load(sbase + sj * p.stage_bytes,
                      p.img + (size_t)(chunk0 + cj) * p.stage_bytes, p.stage_bytes, full(sj));
          }
          __syncwarp();
        }
        ++j;
        if (++cj == nch) cj = 0;
        if (++sj == p.nst) sj = 0, pe ^= 1;
      };
      while (j < p.nst) load_weights();
      for (int i = 0; i < total; ++i) {
        if (ring && j < uses) {
          // the stage used longest ago, when its product is done; this item's weights for certain
          const bool must = j <= i;
          if (must) mbar_wait(empty(sj), pe, failed, status);
          if (must || __all_sync(0xffffffffu, mbar_test(empty(sj), pe))) load_weights();
        }
        if (ring || i < nch) mbar_wait(full(s1), pw, failed, status);
        if (c1 == 0) mbar_wait(x_ready(x1), px, failed, status);
        mbar_wait(gu_free(gu), pg, failed, status);
        fence_after();
        __syncwarp();
        if (elect_one()) {
          const uint32_t d = tmem + gu * kGu;
          const uint32_t a = x_k + x1 * xs, b = w_k + s1 * ss;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < kx)
              mma(d, a + (k >> 2) * kBlk + (k & 3) * 2, b + (k >> 2) * kWBlk + (k & 3) * 2, id_gu,
                  k > 0);
          if (MODE != kFwd) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < ko)
                mma(d + WR, a + y_off + (k >> 2) * kBlk + (k & 3) * 2, b + down_off + k * 128,
                    id_dh, k > 0);
          }
          commit(gu_full(gb));
          if (MODE != kDw && c1 == nch - 1) commit(x_free(x1));
        }
        __syncwarp();
        if (++gu == p.ngu) gu = 0, pg ^= 1;
        if (++gb == gu_bars) gb = 0;
        if (++s1 == p.nst) s1 = 0, pw ^= 1;
        if (++c1 == nch) {
          c1 = 0;
          if (++x1 == p.nx) x1 = 0, px ^= 1;
        }
      }
      // no copy may be in flight when the CTA ends, after a failed wait either
      for (int k = max(0, loads - p.nst); k < loads; ++k)
        mbar_drain(full(k % p.nst), (k / p.nst) & 1, status);
      if (elect_one()) commit(all_done);
      __syncwarp();
    }
  } else if (warp == 2 * kGroupWarps + 1) {
    // ------------------------------------------------------------------------- second products
    if (nt > 0) {
      const uint32_t id_out = MODE == kFwd  ? idesc(BF, p.op, false, false)
                              : MODE == kDx ? idesc(BF, p.dp, false, true)
                                            : idesc(BF, p.dp, true, true);
      const uint32_t id_wy = idesc(BF, p.op, true, true);
      const uint32_t h_k = desc_lo(sbase + h_off, 16), w_k = desc_lo(sbase, 16);
      const uint32_t x_k = desc_lo(sbase + x_off, 16);
      // chunk, hidden operand, rows, weights, output and its parity
      int c2 = 0, hb = 0, x2 = 0, s2 = 0, o2 = 0;
      uint32_t po = 1;  // (the first round of outputs has nobody to wait for)
      for (int i = 0; i < total; ++i) {
        const bool last = c2 == nch - 1;
        mbar_wait(h_ready(i & 1), (i >> 1) & 1, failed, status);
        if (MODE != kDw && c2 == 0) mbar_wait(out_free(o2), po, failed, status);
        fence_after();
        __syncwarp();
        if (elect_one()) {
          const uint32_t h = h_k + hb * (kHBytes >> 4), w = w_k + s2 * ss;
          const bool add = MODE == kDw ? i > 0 : c2 > 0;
          if (MODE == kFwd) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma(acc + o2 * acc_step, h + k * 2, w + down_off + k * 2, id_out, add || k > 0);
          } else if (MODE == kDx) {
#pragma unroll
            for (int k = 0; k < WR / 16; ++k)
              mma(acc + o2 * acc_step, h + (k >> 2) * kBlk + (k & 3) * 2,
                  w - kK + kWMn + k * 128, id_out, add || k > 0);
          } else {
            const uint32_t hm = h - kK + kMn, x = x_k - kK + kMn + x2 * xs;
#pragma unroll
            for (int k = 0; k < 8; ++k) mma(acc, hm + k * 128, x + k * 128, id_out, add || k > 0);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma(acc + acc_step, hm + (GATED ? kBlk : 0) + k * 128, x + y_off + k * 128, id_wy,
                  add || k > 0);
          }
          commit(done(i & 1));
          if (MODE == kDw) commit(x_free(x2));
          if (MODE != kDw && last) commit(out_full(o2));
          if (ring) commit(empty(s2));
          if (i == total - 1) commit(all_done);
        }
        __syncwarp();
        if (++hb == p.nh) hb = 0;
        if (++s2 == p.nst) s2 = 0;
        c2 = last ? 0 : c2 + 1;
        if (last) {
          if (++x2 == p.nx) x2 = 0;
          if (++o2 == p.no) o2 = 0, po ^= 1;
        }
      }
    }
  } else if (warp >= 2 * kGroupWarps + 2) {
    // ------------------------------------------------------------------------- row tiles
    // x_ready counts an arrival of each loader warp, and the bytes of what comes by TMA
    const int tid = threadIdx.x - (2 * kGroupThreads + 64);
    const bool y_too = MODE != kFwd;
    const uint32_t tma_bytes =
        ((p.x.tiled ? nbx : 0) + (y_too && p.dy.tiled ? nby : 0)) * 16384;
    const uint32_t raw = sbase + p.raw_off;
    // tile n's bulk copies on their way (both arrays' bytes on one barrier)
    auto fetch = [&](int n) {
      const long long r0 = ((long long)me + (long long)n * ctas) * kTile;
      const uint8_t *xa, *ya;
      const uint32_t xn = p.x.raw ? raw_span(p.x, r0, p.f.M, xa) : 0;
      const uint32_t yn = y_too && p.dy.raw ? raw_span(p.dy, r0, p.f.M, ya) : 0;
      mbar_expect(raw_full, xn + yn);
      if (xn) bulk_load(raw, xa, xn, raw_full);
      if (yn) bulk_load(raw + p.x.raw, ya, yn, raw_full);
    };
    const bool staged = nt > 0 && (p.x.raw || (y_too && p.dy.raw));
    // The warp that has read a staged tile last starts the next copy: neither waits for the other.
    // A warp stops at its next row tile once a wait of the CTA has failed (places become free then
    // that were not filled), and after a staged tile that did not come: its phase is still open,
    // and the next one's parity would be an older one's.
    int xb = 0, taken = 0, staged_tile = 0;  // staged_tile: the last known to be on its way
    uint32_t pf = 1;  // (the first round is free)
    if (staged && tid == 0) fetch(0);
    for (int n = 0; n < nt; ++n) {
      if (!mbar_wait<true>(x_free(xb), pf, failed, status)) break;
      const long long r0 = ((long long)me + (long long)n * ctas) * kTile;
      const long long rows = p.f.M - r0;
      uint8_t* Xs = smem + x_off + xb * xbytes;
      uint8_t* Ys = Xs + nbx * 16384;
      __syncwarp();
      if (tid == 0 && tma_bytes) {
        mbar_expect_more(x_ready(xb), tma_bytes);
        if (p.x.tiled)
          for (int b = 0; b < nbx; ++b)
            tile_load(smem_addr(Xs) + b * 16384, &x_map, b * 64, (int)r0, x_ready(xb));
        if (y_too && p.dy.tiled)
          for (int b = 0; b < nby; ++b)
            tile_load(smem_addr(Ys) + b * 16384, &dy_map, b * 64, (int)r0, x_ready(xb));
      }
      bool came = true;
      if (staged) {
        came = mbar_wait(raw_full, n & 1, failed, status);
        staged_tile = n;
      }
      auto take = [&](const RowSrc& src, int blocks, uint32_t at, uint8_t* dst) {
        const uint8_t* start;
        if (src.raw && raw_span(src, r0, p.f.M, start)) {
          at += (uint32_t)(src.base + r0 * src.ld - start);
          for (int b = 0; b < blocks; ++b)
            place_staged(at, (int)src.ld, src.cols, b, rows, tid, dst);
        } else {
          for (int b = 0; b < blocks; ++b) place_rows(src, r0, b, rows, tid, dst);
        }
      };
      if (!p.x.tiled) take(p.x, nbx, raw, Xs);
      if (y_too && !p.dy.tiled) take(p.dy, nby, raw + p.x.raw, Ys);
      fence_async_shared();
      __syncwarp();
      // (the second of the two warps to arrive has read the staged tile last)
      if (lane == 0) {
        const bool second = mbar_arrive_pending(x_ready(xb)) == 1;
        if (staged && n + 1 < nt && second && came) {
          asm volatile("fence.acq_rel.cta;" ::: "memory");  // (the other warp's reads)
          fetch(n + 1);
          staged_tile = n + 1;
        }
      }
      if (++xb == p.nx) xb = 0, pf ^= 1;
      ++taken;
      if (!came) break;
    }
    // no copy may be in flight when the CTA ends, after a failed wait either
    for (int n = max(0, taken - p.nx); n < taken; ++n)
      mbar_drain(x_ready(n % p.nx), (n / p.nx) & 1, status);
    // (when the other warp has started one more since, its phase is the one that is waited for)
    staged_tile = __shfl_sync(0xffffffffu, staged_tile, 0);
    if (staged) mbar_drain(raw_full, staged_tile & 1, status);
  } else if (nt > 0) {
    // ------------------------------------------------------------------------- row groups
    const int g = warp / kGroupWarps, tid = threadIdx.x & (kGroupThreads - 1);
    const uint32_t row_lanes = (uint32_t)(warp & 3) << 21;  // 32 * quadrant in the lane field
    const int row = (warp & 3) * 32 + lane, half = (warp >> 2) & 1;
    const bool second = TWICE && half == 1;  // this warp's units are there again
    auto arrive = [&](uint32_t bar) {
      fence_async_shared();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto wait = [&](uint32_t bar, int phase) {
      mbar_wait(bar, phase & 1, failed, status);
      fence_after();
    };
    const float scale = kScaled ? power_of_two(shift) : 1.0f;  // of da and du
    auto group_sync = [&]() {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(kGroupThreads) : "memory");
    };
    auto first_row = [&](int n) { return ((long long)me + (long long)n * ctas) * kTile; };
    // Output of tile n through shared memory to the row array. With a place of their own the groups
    // take them in turn, after their first item of the next tile; else the group of the tile's last
    // item takes it, through the place of that item's hidden operand (whose product is done when the
    // output is complete).
    auto output = [&](int n, int i) {
      const int cols = MODE == kFwd ? p.f.O : p.f.D;
      auto value = [&](uint32_t bits) {  // (dx of scaled da and du)
        return kScaled ? __uint_as_float(bits) * back : __uint_as_float(bits);
      };
      const uint32_t src = acc + (n % p.no) * acc_step + row_lanes + half * 32;
      // (the phase before is over: this group has seen the end of an item behind tile n - no)
      if (p.staged) {
        if (i == total && total >= 2) {  // (the group's last item)
          const int e = (total - 1 - g) / 2 * 2 + g;
          wait(done(e & 1), e >> 1);
        }
        wait(out_full(n % p.no), n / p.no);
      } else {
        wait(done(i & 1), i >> 1);
      }
      uint8_t* S = smem + h_off + p.nh * kHBytes + g * 16384;
      if (!p.staged) S = smem + h_off + (i % p.nh) * kHBytes;
      // Rows of odd widths without gaps: the tile is put together as it lies in memory and leaves as
      // one bulk copy.
      if (p.staged && p.out_dense && first_row(n) + kTile <= p.f.M) {
        if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        group_sync();
        if (half * 32 < cols) {
          uint32_t v0[16], v1[16];
          tmem_ld(src, v0);
          tmem_ld(src + 16, v1);
          tmem_wait(v0);
          tmem_wait(v1);
          uint16_t* q = reinterpret_cast<uint16_t*>(S) + row * cols + half * 32;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint32_t w =
                e < 16 ? Two<T>::pack(value(v0[e & 15]), value(v0[(e + 1) & 15]))
                       : Two<T>::pack(value(v1[e & 15]), value(v1[(e + 1) & 15]));
            if (half * 32 + e < cols) q[e] = (uint16_t)w;
            if (half * 32 + e + 1 < cols) q[e + 1] = (uint16_t)(w >> 16);
          }
        }
        arrive(out_free(n % p.no));
        group_sync();
        if (tid == 0) {
          bulk_store((uint8_t*)(MODE == kFwd ? p.f.y : p.f.dx) + first_row(n) * cols * 2,
                     smem_addr(S), kTile * cols * 2);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        return;
      }
      if (p.staged && p.out_dense) {  // (the last tile: an earlier one may still be leaving)
        if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        group_sync();
      }
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
              const int j = (e + k) & 15;
              w[k / 2] = e < 16 ? Two<T>::pack(value(v0[j]), value(v0[j + 1]))
                                : Two<T>::pack(value(v1[j]), value(v1[j + 1]));
            }
            *reinterpret_cast<uint4*>(S + row * 128 + (((half * 4 + e / 8) ^ (row & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if ((b + 1) * 64 >= cols) {
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(out_free(n % p.no));
        }
        group_sync();
        write_rows(S, (uint8_t*)(MODE == kFwd ? p.f.y : p.f.dx),
                   2 * (MODE == kFwd ? p.f.ldy : p.f.lddx), p.out_aligned, b * 64, cols,
                   first_row(n), p.f.M, tid);
        group_sync();
      }
    };
    // this thread: row `row` of the tile, units half * 32 .. + 32, taken kUnits at a time; the
    // next units' accumulators are on their way while one set is worked on (16 with rests as well
    // would spill: 758,527 rows of 2 / 104 / 21 take 257 us so, 239 with 8)
    constexpr int kUnits = MODE == kFwd && !TWICE ? 16 : 8;
    constexpr int kSteps = 32 / kUnits;
    auto get = [&](uint32_t d, int q, uint32_t (&ra)[kUnits], uint32_t (&ru)[kUnits],
                   uint32_t (&rd)[kUnits]) {
      const uint32_t at = d + half * 32 + q * kUnits;
      tmem_ld(at, ra);
      if (GATED) tmem_ld(at + 64, ru);
      if (MODE != kFwd) tmem_ld(at + WR, rd);
    };
    auto landed = [&](uint32_t (&ra)[kUnits], uint32_t (&ru)[kUnits], uint32_t (&rd)[kUnits]) {
      tmem_wait(ra);
      if (GATED) tmem_wait(ru);
      if (MODE != kFwd) tmem_wait(rd);
    };
    auto work = [&](uint8_t* Hs, int q, const uint32_t (&ra)[kUnits], const uint32_t (&ru)[kUnits],
                    const uint32_t (&rd)[kUnits]) {
      const int piece = half * 4 + q * kUnits / 8;
      if (TWICE && second)
        return hidden_units<MODE, T, ACT, GATED, true, kUnits>(Hs, row, piece, ra, ru, rd, scale);
      return hidden_units<MODE, T, ACT, GATED, false, kUnits>(Hs, row, piece, ra, ru, rd, scale);
    };
    // Sets of four of the thread's 32 units that have to be taken ALONE, from the accumulators once
    // more (a row's results do not depend on the other rows of its warp). Kept out of the other
    // way's registers, where a second look at a set's values would cost 4 to 9 % of the kernel.
    // (A call of 917,504 rows of 64 / 256 / 64, nothing in L2: 191 us with a of deviation 1 to 4, 200
    // with 8, 269 with 15, 324 from 30 on.)
    auto work_alone = [&](uint8_t* Hs, uint32_t d) {
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        uint32_t ra[4], ru[4], rd[4];
        const uint32_t at = d + half * 32 + k * 4;
        tmem_ld(at, ra);
        tmem_wait(ra);
        const float2 a[2] = {make_float2(__uint_as_float(ra[0]), __uint_as_float(ra[1])),
                             make_float2(__uint_as_float(ra[2]), __uint_as_float(ra[3]))};
        float2 f[2], sl[2];
        const bool want = !act4<ACT, false, false>(a, f, sl);
        if (!__any_sync(0xffffffffu, want)) continue;
        if (GATED) tmem_ld(at + 64, ru);
        if (MODE != kFwd) tmem_ld(at + WR, rd);
        if (GATED) tmem_wait(ru);
        if (MODE != kFwd) tmem_wait(rd);
        uint8_t* dst = Hs + row * 128 + (((half * 4 + k / 2) ^ (row & 7)) << 4) + (k & 1) * 8;
        if (TWICE && second)
          hidden_alone<MODE, T, ACT, GATED, true>(dst, want, ra, ru, rd, scale);
        else
          hidden_alone<MODE, T, ACT, GATED, false>(dst, want, ra, ru, rd, scale);
        __syncwarp();
      }
    };

    int c = g, n = 0;
    for (int i = g; i < total; i += 2, c += 2) {
      while (c >= nch) c -= nch, ++n;
      wait(gu_full(i % gu_bars), i / gu_bars);
      const uint32_t d = tmem + (i % p.ngu) * kGu + row_lanes;
      uint8_t* Hs = smem + h_off + (i % p.nh) * kHBytes;
      uint32_t a0[kUnits], u0[kUnits], d0[kUnits], a1[kUnits], u1[kUnits], d1[kUnits];
      get(d, 0, a0, u0, d0);
      // the hidden operand's place was item i - nh's (asked before this item is handed over: the
      // barrier's next phase cannot be complete yet)
      if (i >= p.nh) wait(done((i - p.nh) & 1), (i - p.nh) >> 1);
      bool ok = true;
#pragma unroll
      for (int q = 0; q < kSteps; q += 2) {
        landed(a0, u0, d0);
        get(d, q + 1, a1, u1, d1);
        ok &= work(Hs, q, a0, u0, d0);
        landed(a1, u1, d1);
        if (q + 2 < kSteps) {
          get(d, q + 2, a0, u0, d0);
          ok &= work(Hs, q + 1, a1, u1, d1);
          continue;
        }
        // the accumulators are free once the last values are here, unless some may be asked for
        // again
        auto release = [&]() {
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(gu_free(i % p.ngu));
        };
        if (ACT == SPLAT_ACT_SILU) {
          float least = __uint_as_float(a1[0]);
#pragma unroll
          for (int e = 1; e < kUnits; ++e) least = min_nan(least, __uint_as_float(a1[e]));
          // (two copies of the last units' work: with one, whose result is looked at, the call took
          // 196 us)
          const bool done_with = __all_sync(0xffffffffu, ok && least >= kFar);
          if (done_with) {
            release();
            work(Hs, q + 1, a1, u1, d1);
          } else {
            ok &= work(Hs, q + 1, a1, u1, d1);
            if (!__all_sync(0xffffffffu, ok)) work_alone(Hs, d);
            release();
          }
        } else {
          release();
          work(Hs, q + 1, a1, u1, d1);
        }
      }
      arrive(h_ready(i & 1));
      if (MODE != kDw) {
        // (every group has one item of the first two of a tile; with one chunk, every other tile)
        if (!p.staged) {
          if (c == nch - 1) output(n, i);
        } else if (c < 2 && n > 0 && (nch == 1 || ((n - 1) & 1) == g)) {
          output(n - 1, i);
        }
      }
    }
    if (MODE != kDw && p.staged && (nch == 1 ? g == (nt & 1) : g == ((nt - 1) & 1)))
      output(nt - 1, total);
    // (shared memory is read by the bulk copies until they say so)
    if (MODE != kDw && tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }

  if (MODE == kDw && warp < kGroupWarps) {
    // the CTA's sums: lanes are units (gate, up | up or gate, h), columns D or O
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;
    const uint32_t row_lanes = (uint32_t)(warp & 3) << 21;
    const size_t FD = (size_t)p.f.F * p.f.D;
    constexpr bool two = TWICE;
    float* part = p.f.part + (size_t)(two ? 2 * me + ((row >> 5) & 1) : me) *
                                 ((GATED ? 2 : 1) * FD + (size_t)p.f.F * p.f.O);
    const int f = chunk0 * p.units + (two ? row & 31 : row & 63);
    if (nt > 0) {
      mbar_wait(all_done, 0, failed, status);
      fence_after();
    }
    for (int which = 0; which < 2; ++which) {
      const int cols = which ? p.f.O : p.f.D;
      const bool mine = f < p.f.F && (which ? row >= 64 : GATED || row < 64);
      float* dst = part + (which ? (GATED ? 2 : 1) * FD + (size_t)f * p.f.O
                                 : (row >= 64 ? FD : 0) + (size_t)f * p.f.D);
      // 32 columns at a time: what the launch before left is asked for at once (one after the
      // other, as the stores would have it, a launch took 80 us more)
#pragma unroll 1
      for (int e0 = half * 8; e0 < cols; e0 += 64) {
        float sum[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = e0 + 16 * j + e;
            sum[j][e] = p.again && mine && c < cols ? dst[c] : 0.0f;
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (e0 + 16 * j >= cols) break;
          uint32_t v[8];
          tmem_ld(acc + which * acc_step + row_lanes + e0 + 16 * j, v);
          tmem_wait(v);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (nt > 0)
              sum[j][e] += __uint_as_float(v[e]) * (kScaled && which == 0 ? back : 1.0f);
        }
        if (mine)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e0 + 16 * j + e < cols) dst[e0 + 16 * j + e] = sum[j][e];
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 2 * kGroupWarps) {
    // every MMA is done before TMEM is given back
    if (nt > 0) mbar_drain(all_done, 0, status);
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

// shared memory for a tile as it lies in memory; 0 when the gaps are most of it
int tile_bytes(long long step, int cols) {
  // (place_staged reads up to 20 bytes from a row's last piece)
  const long long b = (step * (kTile - 1) + cols * 2 + 31 + 16) & ~15LL;
  return b <= 2LL * kTile * (cols * 2 + 16) ? (int)((b + 127) & ~127LL) : 0;
}

RowSrc row_src(const void* p, long long ld, long long rows, int cols, CUtensorMap* map,
               CUtensorMapDataType type) {
  RowSrc s = {};
  if (rows <= 0) return s;
  s.base = (const uint8_t*)p;
  s.ld = rows > 1 ? ld * 2 : 0;
  s.cols = cols;
  s.lo = (const uint8_t*)(((uintptr_t)p + 3) & ~(uintptr_t)3);
  s.hi = (const uint8_t*)(((uintptr_t)p + (uintptr_t)((rows - 1) * ld * 2 + cols * 2)) &
                          ~(uintptr_t)3);
  // a tensor map takes 16-byte aligned starts and (positive) distances
  const long long step = rows > 1 ? ld * 2 : (cols * 2 + 15) & ~15;
  s.raw = tile_bytes(step, cols);
  if (((uintptr_t)p & 15) || (step & 15) || step < cols * 2) return s;
  static const auto encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (decltype(&cuTensorMapEncodeTiled))f;
  }();
  if (!encode) return s;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)step};
  const cuuint32_t box[2] = {64, kTile}, unit[2] = {1, 1};
  s.tiled = encode(map, type, 2, const_cast<void*>(p), dims, strides, box, unit,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  return s;
}

int pad16(int v) { return (v + 15) & ~15; }

int stage_bytes(int D, int O, bool gated) {
  return (D + 63) / 64 * (gated ? 128 : 64) * 128 + pad16(O) * 128;
}

// What a CTA keeps in shared memory and TMEM. Two weight stages at least (a ring needs them, unless
// there is one chunk), then as many row tiles and hidden operands as fit, a place for outputs, and
// with the rest more weight stages. Weights mode wants three row tiles, so that a tile's loads wait
// for nothing but the other group's products.
struct Fit {
  int nst, nx, nh, staged, ngu, no, raw_off, smem;
};

Fit fit_of(int mode, bool gated, int dp, int op, int stage, int nch, int raw) {
  static const int kOut[][3] = {{2, 2, 1}, {2, 2, 0}, {1, 2, 1}, {1, 2, 0}};  // nx, nh, staged
  static const int kSum[][3] = {{3, 2, 0}, {2, 2, 0}, {2, 1, 0}, {0, 0, 0}};
  Fit f = {};
  const int gu = gu_cols(mode, gated);
  if (mode == kDw) {
    f.ngu = (512 - pad32(dp) - pad32(op)) / gu;
  } else {
    const int out = pad32(mode == kFwd ? op : dp);
    f.no = (512 - 2 * out) / gu >= 2 ? 2 : 1;
    f.ngu = (512 - f.no * out) / gu;
    if (f.ngu < 2) return Fit{};  // (an output may wait for the item after its own)
  }
  if (f.ngu > kMaxGu) f.ngu = kMaxGu;
  if (f.ngu < 1) return Fit{};
  for (int k = 0; k < 4; ++k) {
    const int* o = mode == kDw ? kSum[k] : kOut[k];
    if (o[0] == 0) break;
    const int used = o[0] * rows_bytes(mode, dp, op) + o[1] * hidden_bytes(mode, gated) +
                     o[2] * 2 * 16384 + raw;  // (outputs: a place for each group)
    const int nst = std::min({(kSmemLimit - used) / stage, nch, kMaxStages});
    if (used > kSmemLimit || nst < std::min(nch, 2)) continue;
    f.nx = o[0];
    f.nh = o[1];
    f.staged = o[2];
    f.nst = nst;
    f.raw_off = nst * stage + used - raw;
    f.smem = nst * stage + used + 1024;
    return f;
  }
  return Fit{};
}

template <int MODE, typename T, int ACT, bool GATED>
int launch(TcArgs p, cudaStream_t st) {
  const bool one = p.f.M <= 1;  // a single row's stride is never used
  CUtensorMap x_map = {}, dy_map = {};
  const auto type =
      Two<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  p.x = row_src(p.f.x, p.f.ldx, p.f.M, p.f.D, &x_map, type);
  if (MODE != kFwd) p.dy = row_src(p.f.dy, p.f.lddy, p.f.M, p.f.O, &dy_map, type);
  if (MODE != kDw) {
    const void* out = MODE == kFwd ? p.f.y : p.f.dx;
    const long long ld = MODE == kFwd ? p.f.ldy : p.f.lddx;
    const int cols = MODE == kFwd ? p.f.O : p.f.D;
    p.out_aligned = aligned16(out, one ? 0 : ld, cols);
    p.out_dense = !p.out_aligned && ld == cols && cols <= 64 && ((uintptr_t)out & 15) == 0;
  }
  const int nch = MODE == kDw ? 1 : p.nch;
  if (p.x.tiled) p.x.raw = 0;
  if (p.dy.tiled) p.dy.raw = 0;
  Fit fit = fit_of(MODE, GATED, p.dp, p.op, p.stage_bytes, nch, p.x.raw + p.dy.raw);
  if (!fit.nst) {
    p.x.raw = p.dy.raw = 0;
    fit = fit_of(MODE, GATED, p.dp, p.op, p.stage_bytes, nch, 0);
  }
  if (!fit.nst) return SPLAT_ERR_CAPACITY;
  p.raw_off = fit.raw_off;
  p.nst = fit.nst;
  p.nx = fit.nx;
  p.nh = fit.nh;
  p.staged = fit.staged;
  p.ngu = fit.ngu;
  p.no = fit.no;
  const long long grid =
      MODE == kDw ? (long long)p.nch * p.f.splits : std::min(p.tiles, 148LL);
  auto kernel = p.units < kChunk ? k_ffn_tc<MODE, T, ACT, GATED, true>
                                 : k_ffn_tc<MODE, T, ACT, GATED, false>;
  // (the same for every launch: the limit is the kernel's, and other host threads set it too)
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemLimit + 1024) != cudaSuccess)
    return SPLAT_ERR_CUDA;
  kernel<<<(unsigned)grid, kTcThreads, fit.smem, st>>>(p, x_map, dy_map);
  return cudaGetLastError() == cudaSuccess ? SPLAT_OK : SPLAT_ERR_CUDA;
}

template <typename T, int ACT, bool GATED>
int run(const FfnArgs& f, bool backward, uint8_t* img, cudaStream_t st) {
  TcArgs p = {};
  p.f = f;
  p.img = img;
  p.units = units(f.D, f.F, f.O);
  p.nch = (f.F + p.units - 1) / p.units;
  p.stage_bytes = stage_bytes(f.D, f.O, GATED);
  p.dp = pad16(f.D);
  p.op = pad16(f.O);
  p.tiles = ((long long)f.M + kTile - 1) / kTile;
  const int pieces = p.nch * (p.stage_bytes >> 4);
  p.pack_ctas = (pieces + 255) / 256;
  if (f.dy_max) p.parts = (int)std::min((f.M + 127LL) / 128, (long long)kMaxParts);
  k_pack<T, GATED><<<p.pack_ctas + p.parts, 256, 0, st>>>(p, img);
  int rc = SPLAT_OK;
  if (!backward) return launch<kFwd, T, ACT, GATED>(p, st);
  if (f.dx && f.M > 0) rc = launch<kDx, T, ACT, GATED>(p, st);
  if (!(f.dwg || f.dwu || f.dwd)) return rc;
  const long long most = sum_rows(Two<T>::kBf16) * f.splits;
  for (long long r = 0; rc == SPLAT_OK && (r == 0 || r < f.M); r += most) {
    p.f.x = (const T*)f.x + r * f.ldx;
    p.f.dy = (const T*)f.dy + r * f.lddy;
    p.f.M = (int)std::min(most, f.M - r);
    p.tiles = ((long long)p.f.M + kTile - 1) / kTile;
    p.f.splits = (int)std::max(1LL, std::min((long long)f.splits, p.tiles));  // (the others' sums stay)
    p.again = r > 0;
    rc = launch<kDw, T, ACT, GATED>(p, st);
  }
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
  const int n = units(D, F, O);
  return (size_t)((F + n - 1) / n) * stage_bytes(D, O, gated);
}

int ffn_tc_splits(long long M, int D, int F, int O) {
  const int n = units(D, F, O), chunks = (F + n - 1) / n;
  const long long tiles = (M + kTile - 1) / kTile, s = 148 / chunks;
  return (int)std::max(1LL, std::min(s, tiles));
}

int ffn_tc_parts(int D, int F, int O) { return twice(D, F, O) ? 2 : 1; }

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
