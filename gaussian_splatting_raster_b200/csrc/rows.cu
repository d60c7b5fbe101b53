// Argument checks shared by the per-row operators.
#include "rows.cuh"

namespace splat {
namespace rows {

static int check_ptr(const void* p, int align, int dev) {
  if (!p || ((uintptr_t)p) % align) return SPLAT_ERR_INVALID_ARG;
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return SPLAT_ERR_INVALID_ARG;
  }
  if (at.type == cudaMemoryTypeManaged) return SPLAT_OK;
  if (at.type != cudaMemoryTypeDevice || at.device != dev) return SPLAT_ERR_INVALID_ARG;
  return SPLAT_OK;
}

// [lo, hi) bytes the array touches
static void extent(const Span& s, uintptr_t& lo, uintptr_t& hi) {
  lo = (uintptr_t)s.p;
  hi = lo + (uintptr_t)(((s.rows - 1) * s.ld + s.cols) * s.elem);
}

static bool share(const Span& a, const Span& b) {
  uintptr_t al, ah, bl, bh;
  extent(a, al, ah);
  extent(b, bl, bh);
  if (ah <= bl || bh <= al) return false;
  // (a single row has no stride of its own: it lies beside the other's rows, or not)
  const long long ld = (a.rows > 1 ? a.ld * a.elem : b.ld * b.elem);
  if (ld != (b.rows > 1 ? b.ld * b.elem : ld) || ld == 0) return true;
  // equal strides: they interleave when the column ranges are apart modulo the stride
  const long long d = (((long long)(bl - al)) % ld + ld) % ld;
  return !(d >= a.cols * a.elem && d + b.cols * b.elem <= ld);
}

int check_spans(const Span* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (s[i].rows <= 0) continue;
    if (!s[i].p || ((uintptr_t)s[i].p) % s[i].elem || s[i].ld < 0 || s[i].ld > kMaxLd)
      return SPLAT_ERR_INVALID_ARG;
    if (s[i].out && s[i].rows > 1 && s[i].ld < s[i].cols) return SPLAT_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i) {
    if (!s[i].out || s[i].rows <= 0) continue;
    for (int j = 0; j < n; ++j)
      if (j != i && s[j].rows > 0 && share(s[i], s[j])) return SPLAT_ERR_INVALID_ARG;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SPLAT_ERR_CUDA;
  }
  for (int i = 0; i < n; ++i) {
    if (s[i].rows <= 0) continue;
    const int rc = check_ptr(s[i].p, s[i].elem, dev);
    if (rc != SPLAT_OK) return rc;
  }
  return SPLAT_OK;
}

}  // namespace rows
}  // namespace splat

extern "C" int splat_rows_status(void* stream) {
  unsigned int a = 0, b = 0;
  if (splat::rows::lookup_status_take(&a, (cudaStream_t)stream) != cudaSuccess ||
      splat::rows::ffn_status_take(&b, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return SPLAT_ERR_CUDA;
  }
  return a | b ? SPLAT_ERR_DEVICE_TIMEOUT : SPLAT_OK;
}
