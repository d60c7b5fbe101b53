// Scaled lookup of table rows by index, and its gradient by sorted indices.
//
//   lookup     out_i = s table[ids_i]            0 <= ids_i < N, a zero row otherwise
//   gradient   dtable_n = s sum_{i: ids_i = n} dout_i
//
// The feature rows of anchors or codebooks that many Gaussians share ("ATSplat": K offsets of one
// anchor) become per-Gaussian rows by the first, and the Gaussians' gradients (the map scatter's
// output, say) return to the shared rows by the second.
//
// The lookup is bound by memory: each output row is written once, each id read once, table rows
// come from L2 where they are shared.
//
// The gradient orders the rows by id (stable LSD radix sort of (id, row) pairs; skipped on the
// device when the ids are in order already, as they are for anchors), then sums each id's run of
// rows in fp32. The order of every sum depends only on the ids, so results are the same bits on
// every run. Work is split over sorted entries, not over table rows: one id may own any share of
// them. A group of lanes that spans one row sums kRun consecutive entries; runs that end inside
// the group are written at once, the rest are joined first within the CTA (shared memory), then
// across CTAs from fp32 partial rows by the finishing kernel, which also zeroes rows nobody uses.
#include "rows.cuh"

namespace splat {
namespace rows {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 32;         // sorted entries one lane group sums
constexpr int kMaxBits = 10;     // digit width of one radix pass
constexpr int kMaxDigits = 1 << kMaxBits;
constexpr int kMaxC = 8192;

template <int VB> struct Bytes;
template <> struct Bytes<2> { using type = uint16_t; };
template <> struct Bytes<4> { using type = uint32_t; };
template <> struct Bytes<8> { using type = uint2; };
template <> struct Bytes<16> { using type = uint4; };

template <typename T, int VB> union Vec {
  static constexpr int N = VB / (int)sizeof(T);
  typename Bytes<VB>::type raw;
  T e[N];
  __device__ Vec() {}
};

// ---------------------------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------------------------

// One CTA: rows [b * rpb, ...), their vectors spread over the threads. magic = ceil(2^32 / vpr)
// divides the CTA-local vector index (< 2^14) by the vectors per row exactly.
template <typename T, int VB>
__global__ void __launch_bounds__(kThreads)
k_lookup(const T* __restrict__ table, long long ldt, unsigned N, const int* __restrict__ ids,
         long long M, int vpr, uint32_t magic, int rpb, float scale, T* __restrict__ out,
         long long ldo) {
  using V = Vec<T, VB>;
  constexpr int U = 4;
  const long long r0 = (long long)blockIdx.x * rpb;
  const int nv = (int)min((long long)rpb, M - r0) * vpr;
  for (int l0 = threadIdx.x; l0 < nv; l0 += kThreads * U) {
    V v[U];
    int row[U], col[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int l = l0 + k * kThreads;
      if (l >= nv) break;
      row[k] = vpr == 1 ? l : (int)__umulhi((uint32_t)l, magic);
      col[k] = (l - row[k] * vpr) * V::N;
      const unsigned id = (unsigned)ids[r0 + row[k]];
#pragma unroll
      for (int e = 0; e < V::N; ++e) v[k].e[e] = from_f<T>(0.0f);
      if (id < N)
        v[k].raw = __ldg(reinterpret_cast<const typename Bytes<VB>::type*>(
            table + (long long)id * ldt + col[k]));
      else
        row[k] = ~row[k];  // a zero row, not scaled: s may be infinite
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (l0 + k * kThreads >= nv) break;
      int r = row[k];
      if (r >= 0) {
#pragma unroll
        for (int e = 0; e < V::N; ++e) v[k].e[e] = from_f<T>(scale * to_f<T>(v[k].e[e]));
      } else {
        r = ~r;
      }
      __stcs(reinterpret_cast<typename Bytes<VB>::type*>(out + (r0 + r) * ldo + col[k]),
             v[k].raw);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// stable order of the ids
// ---------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t key_of(int id, uint32_t N) {
  return (uint32_t)id < N ? (uint32_t)id : N;  // what belongs to no row sorts last
}

// Digit counts of each CTA's items. FIRST: from the ids; also marks CTAs that hold a descent (so
// the order of the ids needs no sort when there is none) and clears the runs' bounds. Later
// passes read pairs and do nothing when the ids were in order.
template <bool FIRST>
__global__ void __launch_bounds__(kThreads)
k_hist(const int* __restrict__ ids, const uint2* __restrict__ pairs, unsigned M, uint32_t N,
       int shift, int bits, unsigned per_block, int* __restrict__ hist, int* __restrict__ descent,
       const int* __restrict__ unsorted, uint2* __restrict__ bounds) {
  __shared__ int cnt[kMaxDigits];
  if (!FIRST && !*unsorted) return;
  const int nd = 1 << bits;
  for (int d = threadIdx.x; d < nd; d += kThreads) cnt[d] = 0;
  __syncthreads();
  const unsigned b = blockIdx.x * per_block, e = min(M, b + per_block);
  int down = 0;
  for (unsigned i = b + threadIdx.x; i < e; i += kThreads) {
    uint32_t k;
    if (FIRST) {
      k = key_of(ids[i], N);
      if (i > 0 && key_of(ids[i - 1], N) > k) down = 1;
    } else {
      k = pairs[i].x;
    }
    atomicAdd(&cnt[(k >> shift) & (nd - 1)], 1);
  }
  if (FIRST) {
    down = __syncthreads_or(down);
    if (threadIdx.x == 0) descent[blockIdx.x] = down;
    for (unsigned n = blockIdx.x * kThreads + threadIdx.x; n < N; n += gridDim.x * kThreads)
      bounds[n] = make_uint2(0u, 0u);
  } else {
    __syncthreads();
  }
  for (int d = threadIdx.x; d < nd; d += kThreads)
    hist[(size_t)d * gridDim.x + blockIdx.x] = cnt[d];
}

// Per digit (one warp each): its counts over the CTAs, scanned in place, and their total. FIRST:
// digit 0's warp also folds the descent marks into the one flag the other kernels read.
template <bool FIRST>
__global__ void __launch_bounds__(kThreads)
k_digit_scan(int* __restrict__ hist, int nblk, int nd, int* __restrict__ total,
             const int* __restrict__ descent, int* __restrict__ unsorted) {
  const int d = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (d >= nd) return;
  if (!FIRST && !*unsorted) return;
  int* h = hist + (size_t)d * nblk;
  int run = 0, any = 0;
  for (int b = 0; b < nblk; b += 32) {
    const int i = b + lane;
    const int c = i < nblk ? h[i] : 0;
    if (FIRST && d == 0 && i < nblk) any |= descent[i];
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    if (i < nblk) h[i] = run + s - c;
    run += __shfl_sync(0xffffffffu, s, 31);
  }
  if (lane == 0) total[d] = run;
  if (FIRST && d == 0) {
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) *unsorted = any;
  }
}

// Stable scatter of one pass. Each warp owns a contiguous part of the CTA's items: its digit
// counts are taken first, then every item's place is its digit's base (digits before, CTAs
// before, warps before) plus its rank among the warp's earlier items of that digit.
template <bool FIRST>
__global__ void __launch_bounds__(kThreads)
k_scatter_pairs(const int* __restrict__ ids, const uint2* __restrict__ in, unsigned M, uint32_t N,
                int shift, int bits, unsigned per_block, const int* __restrict__ hist,
                const int* __restrict__ total, const int* __restrict__ unsorted,
                uint2* __restrict__ out) {
  __shared__ int cnt[kWarps][kMaxDigits];
  __shared__ int wsum[kWarps];
  if (!*unsorted) return;
  const int nd = 1 << bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = threadIdx.x; d < nd * kWarps; d += kThreads) cnt[d / nd][d % nd] = 0;
  __syncthreads();
  const unsigned per_warp = per_block / kWarps;  // a multiple of 32
  const unsigned wb = min(M, blockIdx.x * per_block + warp * per_warp), we = min(M, wb + per_warp);
  for (unsigned i = wb + lane; i < we; i += 32) {
    const uint32_t k = FIRST ? key_of(ids[i], N) : in[i].x;
    atomicAdd(&cnt[warp][(k >> shift) & (nd - 1)], 1);
  }
  __syncthreads();
  // thread t owns digits [t * q, t * q + q): exclusive scan of the digits' totals over the CTA
  const int q = (nd + kThreads - 1) / kThreads;
  const int d0 = threadIdx.x * q;
  int mine = 0;
  for (int d = d0; d < min(nd, d0 + q); ++d) mine += total[d];
  int s = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  int base = s - mine;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  for (int d = d0; d < min(nd, d0 + q); ++d) {
    int at = base + hist[(size_t)d * gridDim.x + blockIdx.x];
    base += total[d];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int c = cnt[w][d];
      cnt[w][d] = at;
      at += c;
    }
  }
  __syncthreads();
  for (unsigned b = wb; b < we; b += 32) {
    const unsigned i = b + lane;
    const bool ok = i < we;
    uint2 kv = make_uint2(0u, 0u);
    if (ok) kv = FIRST ? make_uint2(key_of(ids[i], N), i) : in[i];
    const uint32_t dig = ok ? (kv.x >> shift) & (nd - 1) : (uint32_t)nd + lane;
    const uint32_t peers = __match_any_sync(0xffffffffu, dig);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    int at = 0;
    if (ok) at = cnt[warp][dig] + rank;
    __syncwarp();
    if (ok && rank == 0) cnt[warp][dig] += __popc(peers);
    __syncwarp();
    if (ok) out[at] = kv;
  }
}

// ---------------------------------------------------------------------------------------------
// sums of runs
// ---------------------------------------------------------------------------------------------

struct RunArgs {
  const int* ids;
  const uint2* pairs;
  const int* unsorted;  // 0: entry i is (ids[i], row i); else pairs[i]
  unsigned M;
  uint32_t N;
  int C;
  int gl_log;  // log2 of the lanes per row
  float scale;
  uint2* bounds;  // [N] first and one-past-last sorted entry of each id
  float* head;    // [CTAs][C] part of the run that entered the CTA
  float* tail;    // [CTAs][C] part of the run that leaves it, when it starts in it
};

__device__ __forceinline__ uint2 entry(const RunArgs& a, bool sorted, unsigned i) {
  return sorted ? make_uint2(key_of(a.ids[i], a.N), i) : a.pairs[i];
}

template <typename T, int VB>
__device__ __forceinline__ void put_row(T* dst, const float* acc, float scale) {
  Vec<T, VB> v;
#pragma unroll
  for (int e = 0; e < Vec<T, VB>::N; ++e) v.e[e] = from_f<T>(scale * acc[e]);
  *reinterpret_cast<typename Bytes<VB>::type*>(dst) = v.raw;
}

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads)
k_runs(RunArgs a, const T* __restrict__ dout, long long ldd, T* __restrict__ dtable,
       long long ldt) {
  using V = Vec<T, VB>;
  constexpr int VE = V::N;
  __shared__ float s_head[kThreads * VE], s_tail[kThreads * VE];
  __shared__ uint8_t s_kind[kThreads];  // per group: bit 0 head ends here, bit 1 head passes
                                        // through, bit 2 a run starts and leaves
  const int GL = 1 << a.gl_log, NG = kThreads >> a.gl_log;
  const int g = threadIdx.x >> a.gl_log, gl = threadIdx.x & (GL - 1);
  const int col = (blockIdx.y * GL + gl) * VE;
  const bool act = col < a.C;
  const bool sorted = !*a.unsorted;
  const unsigned blk0 = blockIdx.x * (unsigned)(NG * kRun);
  const unsigned i0 = min(a.M, blk0 + g * kRun), i1 = min(a.M, i0 + kRun);
  const bool mark = gl == 0 && blockIdx.y == 0;
  int kind = 0;
  uint32_t leaving = a.N;  // the id of the run that leaves
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.0f;
  if (i0 < i1) {
    uint32_t cur = entry(a, sorted, i0).x;
    bool head = i0 > 0 && entry(a, sorted, i0 - 1).x == cur;
    if (!head && mark && cur < a.N) a.bounds[cur].x = i0;
    constexpr int U = 4;
    for (unsigned i = i0; i < i1 && cur < a.N; i += U) {
      uint2 kv[U];
      V v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        kv[k] = make_uint2(a.N, 0u);
        if (i + k < i1) kv[k] = entry(a, sorted, i + k);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[k].e[e] = from_f<T>(0.0f);
        if (kv[k].x < a.N && act)
          v[k].raw = __ldcs(reinterpret_cast<const typename Bytes<VB>::type*>(
              dout + (long long)kv[k].y * ldd + col));
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (i + k >= i1) break;
        if (kv[k].x != cur) {  // the run before ended at i + k
          if (cur < a.N) {
            if (head) {
              kind |= 1;
#pragma unroll
              for (int e = 0; e < VE; ++e) s_head[threadIdx.x * VE + e] = acc[e];
            } else if (act) {
              put_row<T, VB>(dtable + (long long)cur * ldt + col, acc, a.scale);
            }
            if (mark) a.bounds[cur].y = i + k;
          }
          cur = kv[k].x;
          head = false;
          if (mark && cur < a.N) a.bounds[cur].x = i + k;
#pragma unroll
          for (int e = 0; e < VE; ++e) acc[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += to_f<T>(v[k].e[e]);
      }
    }
    if (cur < a.N) {
      const bool goes_on = i1 < a.M && entry(a, sorted, i1).x == cur;
      if (!goes_on && mark) a.bounds[cur].y = i1;
      if (head) {
        kind |= goes_on ? 2 : 1;
#pragma unroll
        for (int e = 0; e < VE; ++e) s_head[threadIdx.x * VE + e] = acc[e];
      } else if (goes_on) {
        kind |= 4;
        leaving = cur;
#pragma unroll
        for (int e = 0; e < VE; ++e) s_tail[threadIdx.x * VE + e] = acc[e];
      } else if (act) {
        put_row<T, VB>(dtable + (long long)cur * ldt + col, acc, a.scale);
      }
    }
  }
  if (gl == 0) s_kind[g] = (uint8_t)kind;
  __syncthreads();
  // runs that cross groups: from the group where they start, or from the CTA's first group for
  // the one that entered the CTA
  const bool enters = g == 0 && (kind & 3);
  if (!act) return;
  if (enters) {
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = 0.0f;
    for (int h = 0; h < NG; ++h) {
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += s_head[((h << a.gl_log) + gl) * VE + e];
      if (!(s_kind[h] & 2)) break;
    }
    float* p = a.head + (size_t)blockIdx.x * a.C + col;
#pragma unroll
    for (int e = 0; e < VE; ++e) p[e] = acc[e];
  }
  if (kind & 4) {
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = s_tail[threadIdx.x * VE + e];
    bool open = true;
    for (int h = g + 1; h < NG && open; ++h) {
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += s_head[((h << a.gl_log) + gl) * VE + e];
      open = (s_kind[h] & 2) != 0;
    }
    if (!open) {
      put_row<T, VB>(dtable + (long long)leaving * ldt + col, acc, a.scale);
    } else {
      float* p = a.tail + (size_t)blockIdx.x * a.C + col;
#pragma unroll
      for (int e = 0; e < VE; ++e) p[e] = acc[e];
    }
  }
}

// Rows whose run crosses CTAs (their partial rows summed in order), and zeros for rows without
// entries. A run over more than kLong CTAs is summed by the whole CTA: the groups take equal
// consecutive shares, whose sums are added in order.
constexpr int kLong = 32;

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads)
k_join(RunArgs a, T* __restrict__ dtable, long long ldt) {
  constexpr int VE = Vec<T, VB>::N;
  __shared__ float s_part[kThreads * VE];
  __shared__ uint32_t s_long[kThreads];
  const int GL = 1 << a.gl_log, NG = kThreads >> a.gl_log;
  const int g = threadIdx.x >> a.gl_log, gl = threadIdx.x & (GL - 1);
  const int col = (blockIdx.y * GL + gl) * VE;
  const bool act = col < a.C;
  const unsigned per_cta = NG * kRun;
  const uint32_t n = blockIdx.x * NG + g;
  uint32_t lng = a.N;
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.0f;
  if (n < a.N) {
    const uint2 se = a.bounds[n];
    T* dst = dtable + (long long)n * ldt + col;
    if (se.x == se.y) {
      if (act) put_row<T, VB>(dst, acc, 0.0f);
    } else {
      const unsigned b0 = se.x / per_cta, b1 = (se.y - 1) / per_cta;
      if (b1 - b0 > kLong) {
        lng = n;
      } else if (b1 > b0 && act) {
        const float* p = a.tail + (size_t)b0 * a.C + col;
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] = p[e];
        for (unsigned b = b0 + 1; b <= b1; ++b) {
          const float* h = a.head + (size_t)b * a.C + col;
#pragma unroll
          for (int e = 0; e < VE; ++e) acc[e] += h[e];
        }
        put_row<T, VB>(dst, acc, a.scale);
      }
    }
  }
  if (gl == 0) s_long[g] = lng;
  if (!__syncthreads_or(lng < a.N)) return;
  for (int r = 0; r < NG; ++r) {
    const uint32_t m = s_long[r];
    if (m >= a.N) continue;  // the same for every thread
    const uint2 se = a.bounds[m];
    const unsigned b0 = se.x / per_cta, b1 = (se.y - 1) / per_cta;
    const unsigned share = (b1 - b0 + NG - 1) / NG;
    const unsigned h0 = b0 + 1 + g * share, h1 = min(b1 + 1, h0 + share);
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = 0.0f;
    if (act) {
#pragma unroll 4
      for (unsigned b = h0; b < h1; ++b) {
        const float* h = a.head + (size_t)b * a.C + col;
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += h[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) s_part[threadIdx.x * VE + e] = acc[e];
    __syncthreads();
    if (g == 0 && act) {
      const float* p = a.tail + (size_t)b0 * a.C + col;
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] = p[e];
      for (int h = 0; h < NG; ++h) {
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += s_part[((h << a.gl_log) + gl) * VE + e];
      }
      put_row<T, VB>(dtable + (long long)m * ldt + col, acc, a.scale);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------

// widest access (bytes) that keeps every vector of every row aligned and whole
int vector_bytes(int elem, int C, const void* p, long long ldp, const void* q, long long ldq) {
  const uintptr_t all = (uintptr_t)p | (uintptr_t)q | (uintptr_t)(ldp * elem) |
                        (uintptr_t)(ldq * elem) | (uintptr_t)(C * elem);
  int vb = 16;
  while (vb > elem && (all & (uintptr_t)(vb - 1))) vb >>= 1;
  return vb;
}

struct Plan {
  int passes, bits, nd;
  unsigned per_block, nblk;
  size_t pairs0, pairs1, hist, descent, total, unsorted, bounds, head, tail, bytes;
};

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

Plan make_plan(long long M, long long N, int C) {
  Plan p;
  int need = 1;
  while (need < 32 && (1LL << need) <= N) ++need;  // keys 0 .. N
  p.passes = (need + kMaxBits - 1) / kMaxBits;
  p.bits = (need + p.passes - 1) / p.passes;
  p.nd = 1 << p.bits;
  // enough CTAs for two per SM, at most 8,192 items each
  long long per = (M + 295) / 296;
  per = (per + kThreads - 1) / kThreads * kThreads;
  per = per < kThreads ? kThreads : per > 8192 ? 8192 : per;
  p.per_block = (unsigned)per;
  p.nblk = (unsigned)((M + per - 1) / per);
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o += up(b);
    return at;
  };
  p.pairs0 = take((size_t)M * 8);
  p.pairs1 = take(p.passes > 1 ? (size_t)M * 8 : 0);
  p.hist = take((size_t)p.nd * p.nblk * 4);
  p.descent = take((size_t)p.nblk * 4);
  p.total = take((size_t)p.nd * 4);
  p.unsorted = take(4);
  p.bounds = take((size_t)N * 8);
  const size_t ctas = ((size_t)M + kWarps * kRun - 1) / (kWarps * kRun);  // at 32 lanes a row
  p.head = take(ctas * C * 4);
  p.tail = take(ctas * C * 4);
  p.bytes = o;
  return p;
}

int last_error() {
  return cudaGetLastError() == cudaSuccess ? SPLAT_OK : SPLAT_ERR_CUDA;
}

template <typename T, int VB>
int run_lookup(const T* table, long long ldt, int N, const int* ids, long long M, int C,
               float scale, T* out, long long ldo, cudaStream_t st) {
  const int vpr = C / Vec<T, VB>::N;
  const int rpb = vpr >= 1024 ? 1 : 1024 / vpr;
  const uint32_t magic = (uint32_t)(((1ULL << 32) + vpr - 1) / vpr);
  k_lookup<T, VB><<<(unsigned)((M + rpb - 1) / rpb), kThreads, 0, st>>>(
      table, ldt, (unsigned)N, ids, M, vpr, magic, rpb, scale, out, ldo);
  return last_error();
}

template <typename T, int VB>
int run_sums(RunArgs a, const T* dout, long long ldd, T* dtable, long long ldt, cudaStream_t st) {
  const int vpr = a.C / Vec<T, VB>::N;
  a.gl_log = 0;
  while (a.gl_log < 5 && (1 << a.gl_log) < vpr) ++a.gl_log;
  const int GL = 1 << a.gl_log, NG = kThreads / GL;
  const unsigned cols = (vpr + GL - 1) / GL;
  const unsigned per = NG * kRun;
  k_runs<T, VB><<<dim3((a.M + per - 1) / per, cols), kThreads, 0, st>>>(a, dout, ldd, dtable, ldt);
  k_join<T, VB><<<dim3((a.N + NG - 1) / NG, cols), kThreads, 0, st>>>(a, dtable, ldt);
  return last_error();
}

template <typename T>
int run_backward(const T* dout, long long ldd, const int* ids, long long M, int N, int C,
                 float scale, T* dtable, long long ldt, char* scratch, cudaStream_t st) {
  const Plan p = make_plan(M, N, C);
  int* hist = (int*)(scratch + p.hist);
  int* descent = (int*)(scratch + p.descent);
  int* total = (int*)(scratch + p.total);
  int* unsorted = (int*)(scratch + p.unsorted);
  uint2* bounds = (uint2*)(scratch + p.bounds);
  uint2* buf[2] = {(uint2*)(scratch + p.pairs0), (uint2*)(scratch + p.pairs1)};
  const unsigned m = (unsigned)M, scan_ctas = (p.nd + kWarps - 1) / kWarps;
  for (int i = 0; i < p.passes; ++i) {
    const int shift = i * p.bits;
    uint2* out = buf[i & 1];
    const uint2* in = buf[(i & 1) ^ 1];
    if (i == 0) {
      k_hist<true><<<p.nblk, kThreads, 0, st>>>(ids, nullptr, m, N, shift, p.bits, p.per_block,
                                                hist, descent, unsorted, bounds);
      k_digit_scan<true><<<scan_ctas, kThreads, 0, st>>>(hist, p.nblk, p.nd, total, descent,
                                                         unsorted);
      k_scatter_pairs<true><<<p.nblk, kThreads, 0, st>>>(ids, nullptr, m, N, shift, p.bits,
                                                         p.per_block, hist, total, unsorted, out);
    } else {
      k_hist<false><<<p.nblk, kThreads, 0, st>>>(nullptr, in, m, N, shift, p.bits, p.per_block,
                                                 hist, nullptr, unsorted, nullptr);
      k_digit_scan<false><<<scan_ctas, kThreads, 0, st>>>(hist, p.nblk, p.nd, total, nullptr,
                                                          unsorted);
      k_scatter_pairs<false><<<p.nblk, kThreads, 0, st>>>(nullptr, in, m, N, shift, p.bits,
                                                          p.per_block, hist, total, unsorted, out);
    }
  }
  RunArgs a;
  a.ids = ids;
  a.pairs = buf[(p.passes - 1) & 1];
  a.unsorted = unsorted;
  a.M = m;
  a.N = (uint32_t)N;
  a.C = C;
  a.gl_log = 0;
  a.scale = scale;
  a.bounds = bounds;
  a.head = (float*)(scratch + p.head);
  a.tail = (float*)(scratch + p.tail);
  const int vb = vector_bytes(sizeof(T), C, dout, ldd, dtable, ldt);
  switch (vb) {
    case 16: return run_sums<T, 16>(a, dout, ldd, dtable, ldt, st);
    case 8: return run_sums<T, 8>(a, dout, ldd, dtable, ldt, st);
    case 4: return run_sums<T, 4>(a, dout, ldd, dtable, ldt, st);
  }
  if constexpr (sizeof(T) == 2) return run_sums<T, 2>(a, dout, ldd, dtable, ldt, st);
  return SPLAT_ERR_INVALID_ARG;
}

template <typename T>
int run_forward(const T* table, long long ldt, const int* ids, long long M, int N, int C,
                float scale, T* out, long long ldo, cudaStream_t st) {
  const int vb = vector_bytes(sizeof(T), C, table, ldt, out, ldo);
  switch (vb) {
    case 16: return run_lookup<T, 16>(table, ldt, N, ids, M, C, scale, out, ldo, st);
    case 8: return run_lookup<T, 8>(table, ldt, N, ids, M, C, scale, out, ldo, st);
    case 4: return run_lookup<T, 4>(table, ldt, N, ids, M, C, scale, out, ldo, st);
  }
  if constexpr (sizeof(T) == 2)
    return run_lookup<T, 2>(table, ldt, N, ids, M, C, scale, out, ldo, st);
  return SPLAT_ERR_INVALID_ARG;
}

__global__ void k_zero_rows(char* p, long long row_bytes, long long ld_bytes, long long rows,
                            int unit) {
  const long long per = row_bytes / unit, n = per * rows;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    char* q = p + (i / per) * ld_bytes + (i % per) * unit;
    if (unit == 4) *(uint32_t*)q = 0u;
    else *(uint16_t*)q = 0;
  }
}

}  // namespace
}  // namespace rows
}  // namespace splat

using namespace splat::rows;

extern "C" {

int splat_lookup(const void* table, long long ld_table, int N, int C, const int* ids, int M,
                 float scale, int dtype, void* out, long long ld_out, void* stream) {
  const int es = elem_size(dtype);
  if (!es || N < 0 || M < 0 || C < 1) return SPLAT_ERR_INVALID_ARG;
  if (C > kMaxC) return SPLAT_ERR_CAPACITY;
  if (M == 0) return SPLAT_OK;
  const Span s[] = {{table, N, C, ld_table, es, false},
                    {ids, 1, M, 0, 4, false},
                    {out, M, C, ld_out, es, true}};
  const int rc = check_spans(s, 3);
  if (rc != SPLAT_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  // a single row's stride is never used: it does not limit the access width
  const long long lt = N > 1 ? ld_table : 0, lo = M > 1 ? ld_out : 0;
  if (dtype == SPLAT_F32)
    return run_forward((const float*)table, lt, ids, M, N, C, scale, (float*)out, lo, st);
  if (dtype == SPLAT_BF16)
    return run_forward((const __nv_bfloat16*)table, lt, ids, M, N, C, scale, (__nv_bfloat16*)out,
                       lo, st);
  return run_forward((const __half*)table, lt, ids, M, N, C, scale, (__half*)out, lo, st);
}

long long splat_lookup_scratch(int M, int N, int C) {
  if (M <= 0 || N <= 0 || C < 1 || C > kMaxC) return 0;
  return (long long)make_plan(M, N, C).bytes;
}

int splat_lookup_backward(const void* dout, long long ld_dout, const int* ids, int M, int C,
                          float scale, int dtype, void* dtable, long long ld_dtable, int N,
                          void* scratch, long long scratch_bytes, void* stream) {
  const int es = elem_size(dtype);
  if (!es || N < 0 || M < 0 || C < 1) return SPLAT_ERR_INVALID_ARG;
  if (C > kMaxC) return SPLAT_ERR_CAPACITY;
  if (N == 0) return SPLAT_OK;
  const long long need = splat_lookup_scratch(M, N, C);
  if (scratch_bytes < need) return SPLAT_ERR_INVALID_ARG;
  const Span s[] = {{dout, M, C, ld_dout, es, false},
                    {ids, M ? 1 : 0, M, 0, 4, false},
                    {dtable, N, C, ld_dtable, es, true},
                    {scratch, need ? 1 : 0, need / 16, 0, 16, true}};
  const int rc = check_spans(s, 4);
  if (rc != SPLAT_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  const long long ld = M > 1 ? ld_dout : 0, lt = N > 1 ? ld_dtable : 0;
  if (M == 0) {
    k_zero_rows<<<256, kThreads, 0, st>>>((char*)dtable, (long long)C * es, lt * es, N, es);
    return last_error();
  }
  char* sc = (char*)scratch;
  if (dtype == SPLAT_F32)
    return run_backward((const float*)dout, ld, ids, M, N, C, scale, (float*)dtable, lt, sc, st);
  if (dtype == SPLAT_BF16)
    return run_backward((const __nv_bfloat16*)dout, ld, ids, M, N, C, scale,
                        (__nv_bfloat16*)dtable, lt, sc, st);
  return run_backward((const __half*)dout, ld, ids, M, N, C, scale, (__half*)dtable, lt, sc, st);
}

}  // extern "C"
