// kda_args.h -- host-side argument checks shared by the operators around the prefill: byte ranges
// of dense and strided tensors, their alignment and overlaps.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/kda.h"

namespace kda {

struct ByteRange {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when the tensor is absent
};

inline bool overlap(ByteRange a, ByteRange b) { return a.lo < b.hi && b.lo < a.hi; }

inline ByteRange dense_range(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return p ? ByteRange{lo, lo + bytes} : ByteRange{};
}

inline size_t dtype_bytes(int32_t dtype) { return dtype == KDA_FP32 ? 4 : 2; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks a strided argument over (b, n, s) of the given counts with `row` contiguous elements each
// (1 for a tensor without channels), clears the strides that no index multiplies, and gives the
// range of bytes it covers.
inline kda_status_t check_view(kda_view_t* v, long long nb, long long nn, long long ns, int row,
                               size_t elem, ByteRange* range) {
  if (!v->data) return KDA_ERR_NULL;
  if (nb <= 1) v->stride_b = 0;
  if (nn <= 1) v->stride_n = 0;
  if (ns <= 1) v->stride_s = 0;
  const int64_t st[] = {v->stride_b, v->stride_n, v->stride_s};
  const long long count[] = {nb, nn, ns};
  unsigned long long last = 0;
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || st[i] > (1LL << 46)) return KDA_ERR_SHAPE;
    if (row > 1 && (st[i] * (int64_t)elem) % 16 != 0) return KDA_ERR_ALIGN;
    const __int128 reach = (__int128)st[i] * (count[i] > 0 ? count[i] - 1 : 0);
    if (reach > ((__int128)1 << 56)) return KDA_ERR_SHAPE;
    last += (unsigned long long)reach;
  }
  if (row > 1 ? !aligned16(v->data) : (reinterpret_cast<uintptr_t>(v->data) % elem) != 0)
    return KDA_ERR_ALIGN;
  *range = dense_range(v->data, (size_t)(last + row) * elem);
  return KDA_OK;
}

// Strides of a dense tensor in a layout, over heads N and tokens S with `row` channels.
inline kda_view_t dense_view(const void* p, int32_t layout, long long N, long long S, int row) {
  if (layout == KDA_LAYOUT_BNSD) return {p, N * S * row, S * row, row};
  return {p, S * N * row, row, N * row};  // BSND; TND never multiplies stride_b
}

}  // namespace kda
