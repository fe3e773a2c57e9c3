// kda_recurrence_plan.cpp -- host planner of the gated recurrence: the sequences, longest first, and
// how many steps they take.  Reads lengths only; never touches the GPU.
#include <algorithm>
#include <climits>
#include <cstring>
#include <new>
#include <vector>

#include "kda_recurrence.h"

namespace kda {

kda_status_t validate_recurrence_shape(const kda_recurrence_shape_t* s) {
  if (!s) return KDA_ERR_NULL;
  if (s->layout < KDA_LAYOUT_BNSD || s->layout > KDA_LAYOUT_TND) return KDA_ERR_LAYOUT;
  if (s->D != 128 && s->D != 64) return KDA_ERR_DIM;
  if (s->dtype < KDA_BF16 || s->dtype > KDA_FP32) return KDA_ERR_DTYPE;
  if (s->B < 1 || s->S < 1) return KDA_ERR_SHAPE;
  if (s->N < 1) return KDA_ERR_HEADS;
  const long long rows = s->layout == KDA_LAYOUT_TND ? (long long)s->S : (long long)s->B * s->S;
  if ((long long)s->B * s->N > INT_MAX / 2) return KDA_ERR_SHAPE;
  // rows <= 2^62 and N < 2^31 need a division, not a product, to compare without overflow
  if (rows > (1LL << 46) / s->D / s->N) return KDA_ERR_SHAPE;
  return KDA_OK;
}

namespace {

uint32_t fnv(const int32_t* w, size_t n, uint32_t h = 2166136261u) {
  for (size_t i = 0; i < n; ++i) h = (h ^ (uint32_t)w[i]) * 16777619u;
  return h;
}

// Calls f(b, len) for every sequence of a well-formed problem.
template <class F>
kda_status_t each_length(const kda_recurrence_shape_t& s, const int32_t* cu, F&& f) {
  const bool tnd = s.layout == KDA_LAYOUT_TND;
  if (tnd && !cu) return KDA_ERR_SEQLENS;
  if (cu && (cu[0] != 0 || (tnd && cu[s.B] != s.S))) return KDA_ERR_SEQLENS;
  for (int b = 0; b < s.B; ++b) {
    const long long len = cu ? (long long)cu[b + 1] - cu[b] : s.S;
    if (len < 1 || len > s.S) return KDA_ERR_SEQLENS;
    f(b, (int32_t)len);
  }
  return KDA_OK;
}

long long tiles_of(long long rows, int R) { return (rows + R - 1) / R; }

// Whether the lengths are well formed and everything fits the kernels' 32-bit counters.
kda_status_t check_lengths(const kda_recurrence_shape_t& s, const int32_t* cu) {
  const int R = rec_tile_rows(s.D);
  long long tiles = 0;
  const kda_status_t st = each_length(s, cu, [&](int, int32_t len) {
    tiles += tiles_of(s.layout == KDA_LAYOUT_TND ? len : s.S, R);
  });
  if (st != KDA_OK) return st;
  return tiles > INT_MAX / 2 ? KDA_ERR_SHAPE : KDA_OK;
}

kda_status_t build(const kda_recurrence_shape_t& s, const int32_t* cu, int32_t* plan, size_t n) {
  kda_status_t st = check_lengths(s, cu);
  if (st != KDA_OK) return st;
  if (n < (size_t)kRecHeader + (size_t)s.B * kRecRecord) return KDA_ERR_PLAN;
  const int R = rec_tile_rows(s.D);
  const bool tnd = s.layout == KDA_LAYOUT_TND;
  struct Seq { int32_t b, start, len; };
  std::vector<Seq> seqs;
  seqs.reserve(s.B);
  each_length(s, cu, [&](int b, int32_t len) { seqs.push_back({b, tnd ? cu[b] : 0, len}); });
  std::stable_sort(seqs.begin(), seqs.end(),
                   [](const Seq& a, const Seq& d) { return a.len > d.len; });
  std::memset(plan, 0, kRecHeader * sizeof(int32_t));
  int32_t* rec = plan + kRecHeader;
  long long base = 0, most = 0, steps[kRecClusters] = {};
  for (const Seq& q : seqs) {
    rec[RR_SLOT] = q.b;
    rec[RR_START] = q.start;
    rec[RR_LEN] = q.len;
    rec[RR_BASE] = (int32_t)base;
    rec += kRecRecord;
    base += tiles_of(q.len, R);
    const long long all = tiles_of(tnd ? q.len : s.S, R);
    most = std::max(most, all);
    for (int c = 0; c < kRecClusters; ++c) steps[c] += tiles_of(all, 1 << c);
  }
  plan[RH_MAGIC] = kRecMagic;
  plan[RH_VERSION] = kRecVersion;
  plan[RH_HEADER_WORDS] = kRecHeader;
  plan[RH_RECORD_WORDS] = kRecRecord;
  plan[RH_LAYOUT] = s.layout;
  plan[RH_B] = s.B;
  plan[RH_N] = s.N;
  plan[RH_S] = s.S;
  plan[RH_D] = s.D;
  plan[RH_TILE_ROWS] = R;
  plan[RH_CHAIN] = (int32_t)base;
  plan[RH_MAX_TILES] = (int32_t)most;
  for (int c = 0; c < kRecClusters; ++c) plan[RH_STEPS + c] = (int32_t)steps[c];
  plan[RH_TABLE_HASH] = (int32_t)(fnv(plan + kRecHeader, (size_t)s.B * kRecRecord) & 0x7fffffff);
  plan[RH_CHECKSUM] = (int32_t)(fnv(plan, RH_CHECKSUM) & 0x7fffffff);
  return KDA_OK;
}

}  // namespace

kda_status_t validate_recurrence_plan(const int32_t* p, size_t n, const kda_recurrence_shape_t* s) {
  if (!p) return KDA_ERR_NULL;
  if (n < (size_t)kRecHeader) return KDA_ERR_PLAN;
  if (p[RH_MAGIC] != kRecMagic || p[RH_VERSION] != kRecVersion ||
      p[RH_HEADER_WORDS] != kRecHeader || p[RH_RECORD_WORDS] != kRecRecord)
    return KDA_ERR_PLAN;
  if ((int32_t)(fnv(p, RH_CHECKSUM) & 0x7fffffff) != p[RH_CHECKSUM]) return KDA_ERR_PLAN;
  if (p[RH_B] < 1 || n < (size_t)kRecHeader + (size_t)p[RH_B] * kRecRecord) return KDA_ERR_PLAN;
  if (s && (p[RH_LAYOUT] != s->layout || p[RH_B] != s->B || p[RH_N] != s->N || p[RH_S] != s->S ||
            p[RH_D] != s->D))
    return KDA_ERR_PLAN;
  return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_recurrence_plan_size(const kda_recurrence_shape_t* shape,
                                                 const int32_t* cu, size_t* n_int32) {
  if (!n_int32) return KDA_ERR_NULL;
  kda_status_t st = validate_recurrence_shape(shape);
  if (st != KDA_OK) return st;
  st = check_lengths(*shape, cu);
  if (st != KDA_OK) return st;
  *n_int32 = (size_t)kRecHeader + (size_t)shape->B * kRecRecord;
  return KDA_OK;
}

extern "C" kda_status_t kda_recurrence_plan(const kda_recurrence_shape_t* shape,
                                            const int32_t* cu, int32_t* plan, size_t n_int32) {
  const kda_status_t st = validate_recurrence_shape(shape);
  if (st != KDA_OK) return st;
  if (!plan) return KDA_ERR_NULL;
  try {
    return build(*shape, cu, plan, n_int32);
  } catch (const std::bad_alloc&) {
    return KDA_ERR_SHAPE;
  }
}
