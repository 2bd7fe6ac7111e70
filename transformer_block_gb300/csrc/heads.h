// heads.h — checks of the arguments that the entry points around the block share: views of heads
// (pb_heads), vectors beside them, what they must not overlap; and their tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstdio>

#include "../../include/pb.h"

namespace pb {
pb_status record_error(pb_status s, const char* message);
// Tensor map of one batch entry's heads, [tokens, heads, dh] with the view's strides, read in boxes
// of 64 values x box_heads x box_tokens with 128-byte swizzle (pb_api.cu).
pb_status make_heads_map(CUtensorMap* m, const pb_heads& v, int32_t tokens, int32_t dh,
                         uint32_t box_heads, uint32_t box_tokens);

inline pb_status bad(pb_status s, const char* fmt, const char* what) {
  char msg[200];
  snprintf(msg, sizeof msg, fmt, what);
  return record_error(s, msg);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Dim {
  int64_t n, stride;
};

// Elements from the first to the last value of a view, and its dimensions.
inline int64_t extent(const pb_heads& v, int batch, int seq, int dh, Dim (&d)[3]) {
  d[0] = {batch, v.batch_stride};
  d[1] = {seq, v.seq_stride};
  d[2] = {v.heads, v.head_stride};
  int64_t e = dh;
  for (const Dim& k : d) e += (k.n - 1) * k.stride;
  return e;
}

// Whether no value of the view is another one of it: sorted by stride, each dimension steps
// over all that the smaller ones span.
inline bool distinct(const pb_heads& v, int batch, int seq, int dh) {
  Dim d[3];
  extent(v, batch, seq, dh, d);
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t span = dh;
  for (const Dim& k : d) {
    if (k.n == 1) continue;
    if (k.stride < span) return false;
    span += (k.n - 1) * k.stride;
  }
  return true;
}

inline bool same_view(const pb_heads& a, const pb_heads& b, int batch, int seq) {
  return a.ptr == b.ptr && a.heads == b.heads &&
         (batch == 1 || a.batch_stride == b.batch_stride) &&
         (seq == 1 || a.seq_stride == b.seq_stride) &&
         (a.heads == 1 || a.head_stride == b.head_stride);
}

// Whether two views share no byte, as far as their strides show it: their extents are apart,
// or modulo one of their strides each lies in an interval of its own (the q and k columns of
// one buffer).
inline bool disjoint(const pb_heads& a, const pb_heads& b, int batch, int seq, int dh) {
  Dim da[3], db[3];
  const int64_t ea = extent(a, batch, seq, dh, da), eb = extent(b, batch, seq, dh, db);
  const int64_t pa = int64_t(reinterpret_cast<uintptr_t>(a.ptr)) / 2;
  const int64_t pb_ = int64_t(reinterpret_cast<uintptr_t>(b.ptr)) / 2;
  if (pa + ea <= pb_ || pb_ + eb <= pa) return true;
  for (const Dim& period : da) {
    const int64_t P = period.stride;
    if (period.n < 2 || P <= 0) continue;
    int64_t la = dh, lb = dh;
    for (int k = 0; k < 3; ++k) {
      if (da[k].stride % P != 0) la += (da[k].n - 1) * da[k].stride;
      if (db[k].stride % P != 0) lb += (db[k].n - 1) * db[k].stride;
    }
    if (la > P || lb > P) continue;
    const int64_t gap = ((pb_ - pa) % P + P) % P;  // b's interval behind a's start, mod P
    if (gap >= la && gap + lb <= P) return true;
  }
  return false;
}

// A vector argument beside the views.
struct Flat {
  const void* p;
  size_t bytes;
};

inline bool apart(const Flat& f, const Flat& g) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(f.p), b = reinterpret_cast<uintptr_t>(g.p);
  return f.p == nullptr || g.p == nullptr || a + f.bytes <= b || b + g.bytes <= a;
}
// From the view's first value to its last.
inline bool apart(const Flat& f, const pb_heads* v, int batch, int seq, int dh) {
  if (v == nullptr) return true;
  Dim d[3];
  return apart(f, Flat{v->ptr, size_t(extent(*v, batch, seq, dh, d)) * 2});
}

inline pb_status check_view(const pb_heads* v, const char* what, int batch, int seq, int dh, bool out) {
  if (v->heads < 1) return bad(PB_ERR_INVALID_ARG, "%s: heads must be >= 1", what);
  if (v->ptr == nullptr || !aligned16(v->ptr))
    return bad(PB_ERR_INVALID_ARG, "%s must be a 16-byte aligned device pointer", what);
  const int64_t st[3] = {v->batch_stride, v->seq_stride, v->head_stride};
  for (int64_t k : st)
    if (k < 0 || k % 8 != 0 || k > (int64_t(1) << 40))
      return bad(PB_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements, >= 0", what);
  // so that offsets, in bytes too, and the sums of the checks below stay within 64 bits
  const int64_t steps[3] = {int64_t(batch) - 1, int64_t(seq) - 1, int64_t(v->heads) - 1};
  for (int i = 0; i < 3; ++i)
    if (steps[i] > 0 && st[i] > (int64_t(1) << 48) / steps[i])
      return bad(PB_ERR_UNSUPPORTED, "%s: more than 2^48 values from the first to the last", what);
  if (out && !distinct(*v, batch, seq, dh))
    return bad(PB_ERR_INVALID_ARG, "%s: the strides make values of the result overlap", what);
  return PB_OK;
}

inline pb_status cuda_failed(cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof msg, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return record_error(PB_ERR_CUDA, msg);
}

}  // namespace pb
