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
// come from L2 where they are shared (917,504 rows of 48 fp32 columns out of 4,096: 181 MB in 32.5
// us, 5.6 TB/s; one row 1.5 us, a launch).
//
// The gradient orders the rows by id (stable LSD radix sort of (id, row) pairs; skipped on the
// device when the ids are in order already, as they are for anchors), then sums each id's run of
// rows in fp32. The order of every sum depends only on the ids, so results are the same bits on
// every run. Work is split over sorted entries, not over table rows: one id may own any share of
// them. A group of lanes that spans one row sums up to kRun consecutive entries; runs that end
// inside the group are written at once, the rest are joined first within the CTA (shared memory), then
// across CTAs from fp32 partial rows by the finishing kernel, which also zeroes rows nobody uses.
//
// The sums are bound by memory where rows are read in an order of their own (5.9 M rows of 19 fp16
// columns, 48 bytes apart, by random id: 163 us, 794 MB from DRAM for 224 MB of values, since rows
// share sectors with rows of other ids), the sort by its chain of steps in shared memory (88 us a
// pass at 5.9 M items, 16 at 0.9 M), small calls by their launches (311,296 rows in order: six of 2
// to 10 us).
#include <algorithm>

#include "rows.cuh"

namespace splat {
namespace rows {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 32;         // sorted entries one lane group sums, at most
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

// a row's vector: as one access where it lies inside the array (the elements behind the row's end
// belong to the gap or the next row and are not used), else its n elements
template <typename T, int VB>
__device__ __forceinline__ void get_row(Vec<T, VB>& v, const T* p, int n, const T* end) {
  if (p + Vec<T, VB>::N <= end) {
    v.raw = __ldg(reinterpret_cast<const typename Bytes<VB>::type*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T, VB>::N; ++e) v.e[e] = e < n ? p[e] : from_f<T>(0.0f);
  }
}

// ---------------------------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------------------------

// One CTA: rows [b * rpb, ...), their vectors spread over the threads. magic = ceil(2^32 / vpr)
// divides the CTA-local vector index (< 2^14) by the vectors per row exactly.
template <typename T, int VB>
__global__ void __launch_bounds__(kThreads)
k_lookup(const T* __restrict__ table, long long ldt, unsigned N, const int* __restrict__ ids,
         long long M, int C, int vpr, uint32_t magic, int rpb, float scale, T* __restrict__ out,
         long long ldo) {
  using V = Vec<T, VB>;
  constexpr int U = 4;
  const long long r0 = (long long)blockIdx.x * rpb;
  const T* end = table + (long long)(N - 1) * ldt + C;
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
        get_row<T, VB>(v[k], table + (long long)id * ldt + col[k], C - col[k], end);
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
      T* dst = out + (r0 + r) * ldo + col[k];
      if (col[k] + V::N <= C) {
        __stcs(reinterpret_cast<typename Bytes<VB>::type*>(dst), v[k].raw);
      } else {
#pragma unroll
        for (int e = 0; e < V::N; ++e)
          if (col[k] + e < C) dst[e] = v[k].e[e];
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// stable order of the ids
// ---------------------------------------------------------------------------------------------
// LSD radix sort of (id, row) pairs, digits of up to 10 bits. One kernel reads the ids once for the
// digit totals of every pass and for whether they are in order already; each pass is then one
// kernel of at most 296 CTAs, two to an SM, each with a contiguous share of the items: it counts
// its digits, learns from its predecessors how many of each lie before (look-back: every CTA
// publishes its own counts, and the sum including all before it as soon as it has that), then
// takes its share tile by tile, ranks a tile in shared memory, puts it in digit order there and
// writes runs: 88 us a pass at 5.9 M items. (One tile a CTA would read its items once less, but 720
// CTAs at 5.9 M items then wait for one another in a chain: 123 us a pass.)

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
// most shared memory of a pass: lanes of a digit or the tile, places, counts
constexpr int kSortSmem = 65536 + kMaxDigits * 8 + kSortWarps * kMaxDigits * 2;
static_assert(kSortWarps * kMaxDigits * 4 <= 65536 && kSortThreads * 16 * 8 <= 65536, "");

// how long a CTA waits for its predecessors' counts: about four seconds
#ifndef SPLAT_LOOKUP_WAIT_CLOCKS
#define SPLAT_LOOKUP_WAIT_CLOCKS 8000000000LL
#endif

__device__ unsigned int g_lookup_status;

__device__ __forceinline__ uint32_t key_of(int id, uint32_t N) {
  return (uint32_t)id < N ? (uint32_t)id : N;  // what belongs to no row sorts last
}

struct SortArgs {
  const int* ids;
  uint2 *in, *out;
  unsigned M;
  uint32_t N;
  int pass, passes, bits;
  int vec;              // ids lie at 16 bytes
  uint2* bounds;        // [N] first and one-past-last sorted entry of each id
  // cleared before each call:
  int* total;           // [passes][1 << bits] items of each digit
  int* unsorted;        // whether some id is smaller than the one before it
  unsigned* ticket;     // [passes] CTAs started
  unsigned* state;      // [passes][CTAs][1 << bits] look-back words
  unsigned nblk, share;  // CTAs of a pass, items of one
};

// n pieces of 16 bytes and `tail` 2-byte elements behind them
__global__ void __launch_bounds__(kThreads) k_clear(uint4* p, long long n, int tail) {
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads)
    p[i] = make_uint4(0u, 0u, 0u, 0u);
  if (blockIdx.x == 0 && threadIdx.x < tail)
    reinterpret_cast<uint16_t*>(p + n)[threadIdx.x] = 0;
}

__global__ void __launch_bounds__(kThreads) k_survey(SortArgs a) {
  __shared__ int cnt[3 * kMaxDigits];
  const int nd = 1 << a.bits, n = a.passes * nd;
  for (int d = threadIdx.x; d < n; d += kThreads) cnt[d] = 0;
  __syncthreads();
  int down = 0;
  // threads take 16 consecutive ids at a time (a warp's loads share their lines)
  const unsigned long long stride = (unsigned long long)gridDim.x * kThreads * 16;
  for (unsigned long long i0 = (blockIdx.x * (unsigned long long)kThreads + threadIdx.x) * 16;
       i0 < a.M; i0 += stride) {
    int id[16];
    uint32_t prev = i0 > 0 ? key_of(a.ids[i0 - 1], a.N) : 0u;
    if (a.vec && i0 + 16 <= a.M) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<int4*>(id + 4 * k) =
            __ldg(reinterpret_cast<const int4*>(a.ids + i0) + k);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) id[k] = i0 + k < a.M ? a.ids[i0 + k] : -1;
    }
    const int n = (int)min(16ULL, a.M - i0);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k >= n) break;
      const uint32_t key = key_of(id[k], a.N);
      if (prev > key) down = 1;
      prev = key;
      for (int p = 0; p < a.passes; ++p)
        atomicAdd(&cnt[p * nd + ((key >> (p * a.bits)) & (nd - 1))], 1);
    }
  }
  down = __syncthreads_or(down);
  if (threadIdx.x == 0 && down) *a.unsorted = 1;
  for (int d = threadIdx.x; d < n; d += kThreads)
    if (cnt[d]) atomicAdd(&a.total[d], cnt[d]);
  for (unsigned i = blockIdx.x * kThreads + threadIdx.x; i < a.N; i += gridDim.x * kThreads)
    a.bounds[i] = make_uint2(0u, 0u);
}

// exclusive sum over the CTA of one value per thread
__device__ __forceinline__ int cta_exclusive(int v, int* wsum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  int base = s - v;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  __syncthreads();
  return base;
}

// Look-back words: 0 nothing yet; the CTA's own count plus one; or, with the top bit, the count of
// all CTAs up to and including it (at most 2^31 - 1).
enum : unsigned { kAll = 1u << 31 };

// A few items: CTA 0 sorts them in shared memory (bitonic, on id and row together, so the order is
// stable), the others clear the runs' bounds.
constexpr int kFewItems = 2048;

__global__ void __launch_bounds__(kSortThreads) k_sort_few(SortArgs a, int n) {
  __shared__ unsigned long long s[kFewItems];
  if (blockIdx.x > 0) {
    for (unsigned i = (blockIdx.x - 1) * kSortThreads + threadIdx.x; i < a.N;
         i += (gridDim.x - 1) * kSortThreads)
      a.bounds[i] = make_uint2(0u, 0u);
    return;
  }
  if (threadIdx.x == 0) *a.unsorted = 1;
  for (int i = threadIdx.x; i < n; i += kSortThreads)
    s[i] = i < (int)a.M ? ((unsigned long long)key_of(a.ids[i], a.N) << 32) | (unsigned)i : ~0ULL;
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += kSortThreads) {
        const int i = 2 * t - (t & (j - 1));  // the lower of the pair
        const unsigned long long lo = s[i], hi = s[i + j];
        if ((lo > hi) == ((i & k) == 0)) {
          s[i] = hi;
          s[i + j] = lo;
        }
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < (int)a.M; i += kSortThreads)
    a.out[i] = make_uint2((uint32_t)(s[i] >> 32), (uint32_t)s[i]);
}

// items of a thread and tile: ITEMS, each warp's contiguous, a lane's 32 apart
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads, 2) k_sort_pass(SortArgs a) {
  extern __shared__ __align__(16) int sort_smem[];
  __shared__ int wsum[kSortWarps];
  __shared__ unsigned s_blk;
  if (!*a.unsorted) return;
  const int nd = 1 << a.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shift = a.pass * a.bits;
  constexpr int kItems = kSortThreads * ITEMS;
  uint32_t* mask = reinterpret_cast<uint32_t*>(sort_smem);  // [warps][nd] lanes that hold a digit;
  uint2* sorted = reinterpret_cast<uint2*>(sort_smem);      // then the tile's items in digit order
  int* next = sort_smem + max(kSortWarps * nd, 2 * kItems);  // [nd] global place of the next item
  int* delta = next + nd;                                    // [nd] global minus local place
  uint16_t* cnt = reinterpret_cast<uint16_t*>(delta + nd);   // [warps][nd]
  // CTAs number themselves in the order they start, so those a CTA looks back to have started
  if (threadIdx.x == 0) s_blk = atomicAdd(&a.ticket[a.pass], 1u);
  for (int d = threadIdx.x; d < nd; d += kSortThreads) next[d] = 0;
  __syncthreads();
  const unsigned blk = s_blk;
  const unsigned begin = min(a.M, blk * a.share), end = min(a.M, begin + a.share);
  auto item = [&](unsigned i) {
    return a.pass == 0 ? make_uint2(key_of(a.ids[i], a.N), i) : a.in[i];
  };
#pragma unroll 8
  for (unsigned i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const uint32_t k = a.pass == 0 ? key_of(a.ids[i], a.N) : a.in[i].x;
    atomicAdd(&next[(k >> shift) & (nd - 1)], 1);
  }
  __syncthreads();
  // thread t owns digits [t q, t q + q)
  const int q = (nd + kSortThreads - 1) / kSortThreads;  // 1 or 2
  const int d0 = threadIdx.x * q;
  unsigned* state = a.state + (size_t)a.pass * a.nblk * nd;
  int tot[2] = {0, 0}, own[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int d = d0 + j;
    if (j >= q || d >= nd) continue;
    own[j] = next[d];
    tot[j] = a.total[a.pass * nd + d];
    *(volatile unsigned*)(state + (size_t)blk * nd + d) =
        blk == 0 ? kAll | (unsigned)own[j] : (unsigned)own[j] + 1u;
  }
  const int gbase = cta_exclusive(tot[0] + tot[1], wsum);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int d = d0 + j;
    if (j >= q || d >= nd) continue;
    // items of the digit in earlier CTAs, eight of them asked at a time
    unsigned before = 0;
    const long long t0 = clock64();
    for (unsigned p = blk; p > 0;) {
      unsigned w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        w[k] = p > k ? *(volatile unsigned*)(state + (size_t)(p - 1 - k) * nd + d) : kAll;
      const unsigned asked = p;
      bool done = false;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (done || p != asked - k || w[k] == 0) continue;  // w = 0: not published yet
        if (w[k] & kAll) {
          before += w[k] & ~kAll;
          done = true;
        } else {
          before += w[k] - 1u;
          --p;
        }
      }
      if (done) break;
      if (p == asked && clock64() - t0 > SPLAT_LOOKUP_WAIT_CLOCKS) {
        atomicOr(&g_lookup_status, 1u);
        break;
      }
    }
    if (blk > 0)
      *(volatile unsigned*)(state + (size_t)blk * nd + d) = kAll | (before + (unsigned)own[j]);
    next[d] = gbase + (j ? tot[0] : 0) + (int)before;
  }
  for (unsigned t0 = begin; t0 < end; t0 += kItems) {
    const unsigned n = min((unsigned)kItems, end - t0);
    const unsigned b = t0 + warp * 32 * ITEMS;
    __syncthreads();
    for (int d = threadIdx.x; d < nd * kSortWarps; d += kSortThreads) {
      mask[d] = 0u;
      cnt[d] = 0;
    }
    uint2 kv[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const unsigned i = b + k * 32 + lane;
      kv[k] = make_uint2(0xFFFFFFFFu, 0u);
      if (i < end) kv[k] = item(i);
    }
    __syncthreads();
    // ranks within the warp: a digit's count so far plus the lanes before that hold it too. The
    // lanes find each other through a word per digit (with votes, one per bit, or the match
    // instruction, the pass over 5.9 M items took 114 us instead of 88).
    uint16_t rank[ITEMS];
    uint16_t* mine = cnt + warp * nd;
    uint32_t* lanes = mask + warp * nd;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const bool ok = b + k * 32 + lane < end;
      const uint32_t dig = (kv[k].x >> shift) & (nd - 1);
      if (ok) atomicOr(&lanes[dig], 1u << lane);
      __syncwarp();
      uint32_t peers = 0u, base = 0u;
      if (ok) {
        peers = lanes[dig];
        base = mine[dig];
      }
      const uint32_t before = __popc(peers & ((1u << lane) - 1u));
      __syncwarp();
      if (ok && before == 0) {
        mine[dig] = (uint16_t)(base + __popc(peers));
        lanes[dig] = 0u;
      }
      __syncwarp();
      rank[k] = (uint16_t)(base + before);
    }
    __syncthreads();
    int sum[2] = {0, 0};
    uint16_t c[2][kSortWarps];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int d = d0 + j;
      if (j >= q || d >= nd) continue;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[j][w] = cnt[w * nd + d];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) sum[j] += c[j][w];
    }
    const int lbase = cta_exclusive(sum[0] + sum[1], wsum);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int d = d0 + j;
      if (j >= q || d >= nd) continue;
      int l = lbase + (j ? sum[0] : 0);
      delta[d] = next[d] - l;
      next[d] += sum[j];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {  // a tile has at most 8,192 items
        cnt[w * nd + d] = (uint16_t)l;
        l += c[j][w];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      if (b + k * 32 + lane < end)
        rank[k] = (uint16_t)(rank[k] + mine[(kv[k].x >> shift) & (nd - 1)]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      if (b + k * 32 + lane < end) sorted[rank[k]] = kv[k];
    __syncthreads();
    for (unsigned i = threadIdx.x; i < n; i += kSortThreads) {
      const uint2 v = sorted[i];
      const unsigned at = i + delta[(v.x >> shift) & (nd - 1)];
      if (at < a.M) a.out[at] = v;  // (always, unless a wait ran out)
    }
  }
}

// ---------------------------------------------------------------------------------------------
// sums of runs
// ---------------------------------------------------------------------------------------------

// Entries a lane group sums, one after the other: fewer while 64 groups a CTA (4 lanes a row) would
// leave SMs without one. (The whole gradient at 4,000 rows of 32 fp32 columns, in a graph: 22.5 us,
// with 32 entries always 28.8.)
int run_of(long long M) {
  int run = kRun;
  while (run > 4 && M < 148LL * 64 * run) run >>= 1;
  return run;
}

struct RunArgs {
  const int* ids;
  const uint2* pairs;
  const int* unsorted;  // 0: entry i is (ids[i], row i); else pairs[i]
  unsigned M;
  uint32_t N;
  int C;
  int gl_log;  // log2 of the lanes per row
  int run;     // entries a lane group sums
  float scale;
  uint2* bounds;  // [N] first and one-past-last sorted entry of each id
  float* head;    // [CTAs][C] part of the run that entered the CTA
  float* tail;    // [CTAs][C] part of the run that leaves it, when it starts in it
  int cleared;    // rows without entries are zero already
};

// n of a vector's elements (a row's last vector may be short)
template <typename T, int VB>
__device__ __forceinline__ void put_row(T* dst, const float* acc, float scale, int n) {
  Vec<T, VB> v;
#pragma unroll
  for (int e = 0; e < Vec<T, VB>::N; ++e) v.e[e] = from_f<T>(scale * acc[e]);
  if (n >= Vec<T, VB>::N && ((uintptr_t)dst & (VB - 1)) == 0) {
    *reinterpret_cast<typename Bytes<VB>::type*>(dst) = v.raw;
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T, VB>::N; ++e)
      if (e < n) dst[e] = v.e[e];
  }
}

constexpr int kMinLanes = 4;  // lanes per row at least: bounds the staged entries
constexpr int kMaxEntries = kThreads / kMinLanes * kRun;

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads)
k_runs(RunArgs a, const T* __restrict__ dout, long long ldd, T* __restrict__ dtable,
       long long ldt) {
  using V = Vec<T, VB>;
  constexpr int VE = V::N;
  // the CTA's entries; then, in the same place, the groups' sums of runs that cross them
  __shared__ __align__(16) uint2 s_entry[kMaxEntries + 2];
  static_assert(sizeof(s_entry) >= 2 * kThreads * VE * sizeof(float), "");
  __shared__ uint8_t s_kind[kThreads / kMinLanes];  // per group: bit 0 head ends here, bit 1 head
                                                    // passes through, bit 2 a run starts and leaves
  const int GL = 1 << a.gl_log, NG = kThreads >> a.gl_log;
  const int g = threadIdx.x >> a.gl_log, gl = threadIdx.x & (GL - 1);
  const int col = (blockIdx.y * GL + gl) * VE;
  const int left = a.C - col;  // elements of the row from here on
  const bool act = left > 0;
  const bool sorted = !*a.unsorted;
  const unsigned blk0 = blockIdx.x * (unsigned)(NG * a.run);
  const int count = (int)min((unsigned)(NG * a.run), a.M - blk0);
  // entries blk0 - 1 .. blk0 + count: entry i of the CTA is s_entry[i + 1]
  for (int i = threadIdx.x; i < count + 2; i += kThreads) {
    uint2 kv = make_uint2(0xFFFFFFFFu, 0u);  // no id
    const long long j = (long long)blk0 + i - 1;
    if (j >= 0 && j < a.M)
      kv = sorted ? make_uint2(key_of(a.ids[j], a.N), (uint32_t)j) : a.pairs[j];
    if (kv.y >= a.M) kv.x = a.N;  // (only when a wait of the sort ran out)
    s_entry[i] = kv;
  }
  __syncthreads();
  const T* end = dout + (long long)(a.M - 1) * ldd + a.C;
  const int i0 = min(count, g * a.run), i1 = min(count, i0 + a.run);
  const bool mark = gl == 0 && blockIdx.y == 0;
  int kind = 0;
  uint32_t leaving = a.N;  // the id of the run that leaves
  float acc[VE], first[VE];  // the run at hand; the one that entered, once it ended
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = first[e] = 0.0f;
  if (i0 < i1) {
    uint32_t cur = s_entry[i0 + 1].x;
    bool head = s_entry[i0].x == cur;
    if (!head && mark && cur < a.N) a.bounds[cur].x = blk0 + i0;
    constexpr int U = VB == 16 ? 4 : 8;
    for (int i = i0; i < i1 && cur < a.N; i += U) {
      uint32_t key[U];
      V v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const uint2 kv = s_entry[min(i + k, i1 - 1) + 1];
        key[k] = kv.x;
#pragma unroll
        for (int e = 0; e < VE; ++e) v[k].e[e] = from_f<T>(0.0f);
        if (i + k < i1 && kv.x < a.N && act)
          get_row<T, VB>(v[k], dout + (long long)kv.y * ldd + col, left, end);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (i + k >= i1) break;
        if (key[k] != cur) {  // the run before ended at i + k
          if (cur < a.N) {
            if (head) {
              kind |= 1;
#pragma unroll
              for (int e = 0; e < VE; ++e) first[e] = acc[e];
            } else if (act) {
              put_row<T, VB>(dtable + (long long)cur * ldt + col, acc, a.scale, left);
            }
            if (mark) a.bounds[cur].y = blk0 + i + k;
          }
          cur = key[k];
          head = false;
          if (mark && cur < a.N) a.bounds[cur].x = blk0 + i + k;
#pragma unroll
          for (int e = 0; e < VE; ++e) acc[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += to_f<T>(v[k].e[e]);
      }
    }
    if (cur < a.N) {
      const bool goes_on = s_entry[i1 + 1].x == cur;
      if (!goes_on && mark) a.bounds[cur].y = blk0 + i1;
      if (head) {
        kind |= goes_on ? 2 : 1;
#pragma unroll
        for (int e = 0; e < VE; ++e) first[e] = acc[e];
      } else if (goes_on) {
        kind |= 4;
        leaving = cur;
      } else if (act) {
        put_row<T, VB>(dtable + (long long)cur * ldt + col, acc, a.scale, left);
      }
    }
  }
  __syncthreads();
  float* s_head = reinterpret_cast<float*>(s_entry);
#pragma unroll
  for (int e = 0; e < VE; ++e) s_head[threadIdx.x * VE + e] = first[e];
  if (gl == 0) s_kind[g] = (uint8_t)kind;
  __syncthreads();
  // runs that cross groups: from the group where they start, or from the CTA's first group for
  // the one that entered the CTA
  if (!act) return;
  const int n = min(left, VE);
  if (g == 0 && (kind & 3)) {
    float sum[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) sum[e] = 0.0f;
    for (int h = 0; h < NG; ++h) {
#pragma unroll
      for (int e = 0; e < VE; ++e) sum[e] += s_head[((h << a.gl_log) + gl) * VE + e];
      if (!(s_kind[h] & 2)) break;
    }
    float* p = a.head + (size_t)blockIdx.x * a.C + col;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (e < n) p[e] = sum[e];
  }
  if (kind & 4) {
    bool open = true;
    for (int h = g + 1; h < NG && open; ++h) {
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += s_head[((h << a.gl_log) + gl) * VE + e];
      open = (s_kind[h] & 2) != 0;
    }
    if (!open) {
      put_row<T, VB>(dtable + (long long)leaving * ldt + col, acc, a.scale, left);
    } else {
      float* p = a.tail + (size_t)blockIdx.x * a.C + col;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (e < n) p[e] = acc[e];
    }
  }
}

// Rows whose run crosses CTAs (their partial rows summed in order), and zeros for rows without
// entries: a group a row. In a cleared table only the first are left, at most one a boundary
// between CTAs: a group a boundary, which takes the run that first crosses it. A run over more than
// kLong CTAs is summed by the whole CTA: the groups take equal consecutive shares, whose sums are
// added in order.
constexpr int kLong = 32;

// The entries of row n. Nothing where its bounds do not fit together, as when a wait of the sort
// ran out and the entries are in no order: CTAs are told from them.
__device__ __forceinline__ uint2 entries_of(const RunArgs& a, uint32_t n) {
  const uint2 se = a.bounds[n];
  return se.x < se.y && se.y <= a.M ? se : make_uint2(0u, 0u);
}

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads)
k_join(RunArgs a, T* __restrict__ dtable, long long ldt) {
  constexpr int VE = Vec<T, VB>::N;
  __shared__ float s_part[kThreads * VE];
  __shared__ uint32_t s_long[kThreads / kMinLanes];
  const int GL = 1 << a.gl_log, NG = kThreads >> a.gl_log;
  const int g = threadIdx.x >> a.gl_log, gl = threadIdx.x & (GL - 1);
  const int col = (blockIdx.y * GL + gl) * VE;
  const int left = a.C - col, cnt = min(left, VE);
  const bool act = left > 0;
  const unsigned per_cta = NG * a.run;
  uint32_t n = blockIdx.x * NG + g;
  if (a.cleared) {
    const long long i = ((long long)n + 1) * per_cta;
    uint32_t key = a.N;
    if (i < a.M) key = *a.unsorted == 0 ? key_of(a.ids[i], a.N) : a.pairs[i].x;
    n = key < a.N && a.bounds[key].x / per_cta == n ? key : a.N;
  }
  uint32_t lng = a.N;
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.0f;
  if (n < a.N) {
    const uint2 se = entries_of(a, n);
    T* dst = dtable + (long long)n * ldt + col;
    if (se.x == se.y) {
      if (act) put_row<T, VB>(dst, acc, 0.0f, left);
    } else {
      const unsigned b0 = se.x / per_cta, b1 = (se.y - 1) / per_cta;
      if (b1 - b0 > kLong) {
        lng = n;
      } else if (b1 > b0 && act) {
        const float* p = a.tail + (size_t)b0 * a.C + col;
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] = e < cnt ? p[e] : 0.0f;
        for (unsigned b = b0 + 1; b <= b1; ++b) {
          const float* h = a.head + (size_t)b * a.C + col;
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (e < cnt) acc[e] += h[e];
        }
        put_row<T, VB>(dst, acc, a.scale, left);
      }
    }
  }
  if (gl == 0) s_long[g] = lng;
  if (!__syncthreads_or(lng < a.N)) return;
  for (int r = 0; r < NG; ++r) {
    const uint32_t m = s_long[r];
    if (m >= a.N) continue;  // the same for every thread
    const uint2 se = entries_of(a, m);
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
        for (int e = 0; e < VE; ++e)
            if (e < cnt) acc[e] += h[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) s_part[threadIdx.x * VE + e] = acc[e];
    __syncthreads();
    if (g == 0 && act) {
      const float* p = a.tail + (size_t)b0 * a.C + col;
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] = e < cnt ? p[e] : 0.0f;
      for (int h = 0; h < NG; ++h) {
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += s_part[((h << a.gl_log) + gl) * VE + e];
      }
      put_row<T, VB>(dtable + (long long)m * ldt + col, acc, a.scale, left);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------

// widest access (bytes) that keeps every vector of every row aligned (a row's last may be short)
int vector_bytes(int elem, const void* p, long long ldp, const void* q, long long ldq) {
  const uintptr_t all = (uintptr_t)p | (uintptr_t)q | (uintptr_t)(ldp * elem) |
                        (uintptr_t)(ldq * elem);
  int vb = 16;
  while (vb > elem && (all & (uintptr_t)(vb - 1))) vb >>= 1;
  return vb;
}

struct Plan {
  int passes, bits, nd, items;
  unsigned nblk, share;
  size_t clear, pairs0, pairs1, total, unsorted, ticket, state, bounds, head, tail, bytes;
};

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

Plan make_plan(long long M, long long N, int C) {
  Plan p;
  int need = 1;
  while (need < 32 && (1LL << need) <= N) ++need;  // keys 0 .. N
  p.passes = (need + kMaxBits - 1) / kMaxBits;
  p.bits = (need + p.passes - 1) / p.passes;
  p.nd = 1 << p.bits;
  // tiles of 8,192 items, or of 2,048 while that leaves SMs without one; as many to a CTA as keep
  // the CTAs at two an SM
  p.items = M > 8192LL * 148 ? 16 : 4;
  const long long tile = (long long)kSortThreads * p.items, tiles = (M + tile - 1) / tile;
  const long long per = (tiles + 295) / 296;
  p.share = (unsigned)std::min(per * tile, 1LL << 31);
  p.nblk = (unsigned)((tiles + per - 1) / per);
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o += up(b);
    return at;
  };
  // cleared at the start of a call
  p.total = take((size_t)p.passes * p.nd * 4);
  p.unsorted = take(4);
  p.ticket = take((size_t)p.passes * 4);
  p.state = take((size_t)p.passes * p.nblk * p.nd * 4);
  p.clear = o;
  p.pairs0 = take((size_t)M * 8);
  p.pairs1 = take(p.passes > 1 ? (size_t)M * 8 : 0);
  p.bounds = take((size_t)N * 8);
  const size_t some = kWarps * run_of(M), ctas = ((size_t)M + some - 1) / some;  // at 32 lanes a row
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
  const int vpr = (C + Vec<T, VB>::N - 1) / Vec<T, VB>::N;
  const int rpb = vpr >= 1024 ? 1 : 1024 / vpr;
  const uint32_t magic = (uint32_t)(((1ULL << 32) + vpr - 1) / vpr);
  k_lookup<T, VB><<<(unsigned)((M + rpb - 1) / rpb), kThreads, 0, st>>>(
      table, ldt, (unsigned)N, ids, M, C, vpr, magic, rpb, scale, out, ldo);
  return last_error();
}

template <typename T, int VB>
int run_sums(RunArgs a, const T* dout, long long ldd, T* dtable, long long ldt, cudaStream_t st) {
  const int vpr = (a.C + Vec<T, VB>::N - 1) / Vec<T, VB>::N;
  a.gl_log = 2;
  while (a.gl_log < 5 && (1 << a.gl_log) < vpr) ++a.gl_log;
  const int GL = 1 << a.gl_log, NG = kThreads / GL;
  const unsigned cols = (vpr + GL - 1) / GL;
  const unsigned per = NG * a.run;
  k_runs<T, VB><<<dim3((a.M + per - 1) / per, cols), kThreads, 0, st>>>(a, dout, ldd, dtable, ldt);
  const unsigned groups = a.cleared ? (a.M - 1) / per : a.N;
  if (groups > 0)
    k_join<T, VB><<<dim3((groups + NG - 1) / NG, cols), kThreads, 0, st>>>(a, dtable, ldt);
  return last_error();
}

template <typename T>
int run_backward(const T* dout, long long ldd, const int* ids, long long M, int N, int C,
                 float scale, T* dtable, long long ldt, char* scratch, cudaStream_t st) {
  const Plan p = make_plan(M, N, C);
  SortArgs q;
  q.ids = ids;
  q.vec = ((uintptr_t)ids & 15) == 0;
  q.M = (unsigned)M;
  q.N = (uint32_t)N;
  q.passes = p.passes;
  q.bits = p.bits;
  q.bounds = (uint2*)(scratch + p.bounds);
  q.total = (int*)(scratch + p.total);
  q.unsorted = (int*)(scratch + p.unsorted);
  q.ticket = (unsigned*)(scratch + p.ticket);
  q.state = (unsigned*)(scratch + p.state);
  q.nblk = p.nblk;
  q.share = p.share;
  uint2* buf[2] = {(uint2*)(scratch + p.pairs0), (uint2*)(scratch + p.pairs1)};
  if (M <= kFewItems) {
    int n = 2;
    while (n < M) n <<= 1;
    q.out = buf[(p.passes - 1) & 1];
    const int clear = std::min((N + kSortThreads - 1) / kSortThreads, 296);
    k_sort_few<<<1 + clear, kSortThreads, 0, st>>>(q, n);
  } else {
    const long long words = (long long)(p.clear / 16);
    k_clear<<<(unsigned)std::min((words + kThreads - 1) / kThreads, 148LL * 8), kThreads, 0, st>>>(
        (uint4*)scratch, words, 0);
    const long long want = (std::max(M, (long long)N) + kThreads * 16 - 1) / (kThreads * 16);
    k_survey<<<(unsigned)std::min(want, 148LL * 4), kThreads, 0, st>>>(q);
    const int smem = std::max(kSortWarps * p.nd * 4, kSortThreads * p.items * 8) + p.nd * 8 +
                     kSortWarps * p.nd * 2;
    auto pass = p.items == 16 ? k_sort_pass<16> : k_sort_pass<4>;
    // (the same for every launch: the limit is the kernel's, and other host threads set it too)
    if (cudaFuncSetAttribute(pass, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem) !=
        cudaSuccess)
      return last_error();
    for (int i = 0; i < p.passes; ++i) {
      q.pass = i;
      q.in = buf[(i & 1) ^ 1];
      q.out = buf[i & 1];
      pass<<<p.nblk, kSortThreads, smem, st>>>(q);
    }
  }
  RunArgs a;
  a.ids = ids;
  a.pairs = buf[(p.passes - 1) & 1];
  a.unsorted = q.unsorted;
  a.M = (unsigned)M;
  a.N = (uint32_t)N;
  a.C = C;
  a.gl_log = 0;
  a.run = run_of(M);
  a.scale = scale;
  a.bounds = q.bounds;
  a.head = (float*)(scratch + p.head);
  a.tail = (float*)(scratch + p.tail);
  // A dense table most of whose rows get nothing is cleared first, in 16-byte stores whatever its
  // rows' width (210,142 rows of 323, three entries: 192 us by rows, 48 so).
  a.cleared = 0;
  const size_t bytes = (size_t)N * C * sizeof(T);
  if ((ldt == C || N == 1) && N / 2 > M && ((uintptr_t)dtable & 15) == 0) {
    const long long pieces = (long long)(bytes / 16);
    k_clear<<<(unsigned)std::min(pieces / kThreads + 1, 148LL * 16), kThreads, 0, st>>>(
        (uint4*)dtable, pieces, (int)(bytes % 16) / 2);
    a.cleared = 1;
  }
  const int vb = vector_bytes(sizeof(T), dout, ldd, dout, ldd);
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
  const int vb = vector_bytes(sizeof(T), table, ldt, out, ldo);
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

cudaError_t lookup_status_take(unsigned int* out, cudaStream_t st) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_lookup_status, sizeof *out, 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_lookup_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice,
                                st);
  return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

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
